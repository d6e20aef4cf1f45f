// Launchers of the MXFP4 kernels: quantisation (mx_quant.hip), the dispatch for up to
// 256 experts (mx_dispatch.hip) and the expert products (mx_ffn.hip,
// mx_tile.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace moe {

constexpr int kMxMaxExperts = 256;

hipError_t launch_mx_quantize(const void* x, bool bf16, int64_t rows, int64_t cols, int64_t stride,
                              uint8_t* codes, uint8_t* scales, hipStream_t s);
hipError_t launch_mx_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows,
                                int64_t cols, bool bf16, void* out, int64_t stride, hipStream_t s);
// bf16 rows through MXFP4 and back (the values the 4-bit activations stand for).
hipError_t launch_mx_requantize(const void* x, int64_t rows, int64_t cols, void* out, hipStream_t s);

int mx_dispatch_blocks(int assignments);
struct MxDispatchArgs {
  const int32_t* topk_idx;
  int A, E;                // assignments T*k
  int32_t *counts, *offsets, *dest, *src;
  int32_t *blk_hist, *blk_base;   // [mx_dispatch_blocks(A)][E], used past one block
};
hipError_t launch_mx_dispatch(const MxDispatchArgs& a, hipStream_t s);

struct MxFfnArgs {
  bool up;                 // GELU, bf16 out; else fp32 out
  bool fp4;                // activations in MXFP4
  const void* a;           // bf16 activations
  int64_t a_rows;          // rows of `a`
  const int32_t* src;      // or null; row r reads a[src[r] / k]
  const int32_t* offsets;
  const uint8_t* w;        // [E][N][K/2]
  const uint8_t* ws;       // [E][N][K/32]
  const void* bias;        // [E][N] bf16 or null
  void* out;               // [R][N]
  int T, k, E, N, K;
  uint8_t* act;            // workspace of mx_act_bytes
  float* partial;          // workspace of mx_partial_bytes
};
size_t mx_act_bytes(int T, int k, int E, int N, int K, bool fp4);
size_t mx_partial_bytes(int T, int k, int E, int N, int K);
hipError_t launch_mx_ffn(const MxFfnArgs& a, hipStream_t s);
// mx_tile.hip: the LDS-tiled products (K >= 512).
hipError_t launch_mx_tile(const MxFfnArgs& a, hipStream_t s);
size_t mx_tile_bytes(long rows, int E, int N, int K, bool fp4);

}  // namespace moe
