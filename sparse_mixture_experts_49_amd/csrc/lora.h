// Launchers of the shared projection with low-rank adapters (lora.hip, lora_tile.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace moe {

constexpr int kLoraMaxRank = 128, kLoraMaxAdapters = 4096;

struct LoraShape {
  int T, d, n, rank, N;
  bool gelu, f32_out;
};

// Bytes of workspace: the adapters' first products u, and parts of sums.
size_t lora_u_bytes(const LoraShape& s);

struct LoraArgs {
  LoraShape sh;
  const uint16_t* x;          // [T][d]
  const int32_t* adapter;     // [T]
  const uint16_t* w;          // [n][d]
  const uint16_t* bias;       // [n] or null
  const uint16_t* a;          // [N][rank][d]
  const uint16_t* b;          // [N][n][rank]
  const float* scale;         // [N] or null
  void* y;                    // [T][n] bf16 or fp32
  void* u;                    // workspace of lora_u_bytes
};
hipError_t launch_lora(const LoraArgs& a, hipStream_t s);

// Parts of the k range: fp32 sums for lora_finish_kernel.
struct LoraPartArgs {
  LoraArgs a;
  int splits, a_tiles;                 // parts of k; column tiles that A can have per row tile
  float* part;                         // [splits][T][n]
  float* u;                            // [splits][T][lora_pitch], not scaled
};
void launch_lora_part_tile(const LoraPartArgs& p, unsigned grid, hipStream_t s);   // 128 x 128 tiles

// The tiled product (lora_tile.hip).  u is `lora_terms` bf16 matrices [T][lora_pitch] that add up
// to scale A x.
__host__ __device__ inline int lora_pitch(int rank) { return (rank + 15) / 16 * 16; }
inline int lora_terms(const LoraShape& s) { return s.f32_out ? 3 : 2; }
hipError_t launch_lora_tile(const LoraArgs& a, hipStream_t s);

}  // namespace moe
