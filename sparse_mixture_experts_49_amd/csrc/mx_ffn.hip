// Grouped expert products with MXFP4 weights on gfx950.
//
// out[r] = a[r] W_e^T + b_e for the rows of expert e's segment, W_e [N][K] as e2m1 codes
// with one e8m0 scale per 32 values of k; the first product applies the exact-erf GELU.
#include <algorithm>
#include <type_traits>

#include "device_common.h"
#include "mx.h"

namespace moe {

// Expert e's rows, cut to [0, rows).
__device__ __forceinline__ void segment(const int32_t* __restrict__ offsets, int e, int rows,
                                        int& lo, int& hi) {
  lo = min(max(offsets[e], 0), rows);
  hi = min(max(offsets[e + 1], lo), rows);
}

// Row of the activations that dispatched row r reads.
__device__ __forceinline__ int act_row(const int32_t* __restrict__ src, int k, int tokens, int r) {
  if (!src) return r;
  return (int)min((uint32_t)src[r] / (uint32_t)k, (uint32_t)tokens - 1u);
}

// global -> LDS, 16 bytes per lane to lds_addr + lane * 16 (uniform address); the compiler
// sees no LDS write, so the caller waits for vmcnt itself.
__device__ __forceinline__ void dma16(const void* g, uint32_t lds_addr) {
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off"
               :: "v"(g), "s"(lds_addr) : "memory", "m0");
}

// ---------------------------------------------------------------------------
// Weight streaming (few rows per expert: bound by the bytes of the codes).
//
// Block = 8 waves; wave w owns 16 NW output columns and reads their code rows straight
// into registers: lane (n = l % 16, q = l / 16) takes 16 bytes = one scale block
// of row n, so one load covers 128 k of 16 rows, and each code and scale is read once.
// The block's 16 NMT rows of activations (bf16) go through LDS in chunks of 512 k,
// a ring of kDepth stages filled by DMA; pieces of 16 B of a row sit at piece ^ (row %
// 16) within each 256 B, so a fragment read (16 rows, same piece) touches every bank
// once.  Codes are widened to bf16 by v_cvt_scalef32_pk_bf16_fp4 (exact) and
// multiplied by MFMA 16x16x32; slice s of a 128-k granule takes k = 32 q + 8 s .. + 7
// from both operands.  With `splits` > 1 a block sums one part of k into `partial`.
// ---------------------------------------------------------------------------
constexpr int kStreamWaves = 8, kStreamNW = 2;
constexpr int kStreamCols = kStreamWaves * kStreamNW * 16;
constexpr int kStreamDepth = 3;

template <bool UP, int NMT>
__global__ __launch_bounds__(512) void mx_stream_kernel(
    const uint16_t* __restrict__ A, const int32_t* __restrict__ src, int k_top, int tokens,
    const int32_t* __restrict__ offsets, int rows_cap, const uint8_t* __restrict__ W,
    const uint8_t* __restrict__ WS, const uint16_t* __restrict__ bias, void* __restrict__ out,
    int N, int K, int splits, float* __restrict__ partial) {
  constexpr int kRows = 16 * NMT, NW = kStreamNW;
  constexpr int kStage = kRows * 1024;
  constexpr int kDma = kRows / kStreamWaves;        // 1 KB row pieces per wave per chunk
  __shared__ __attribute__((aligned(1024))) uint8_t lds[kStreamDepth * kStage];

  const int e = blockIdx.y, split = blockIdx.z % splits, groups = gridDim.z / splits;
  int lo, hi;
  segment(offsets, e, rows_cap, lo, hi);
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int fr = lane & 15, fc = lane >> 4;
  const int n0 = blockIdx.x * kStreamCols + wave * 16 * NW;
  const int granules = K / 128;
  const int g0 = (int)((long)split * granules / splits), g1 = (int)((long)(split + 1) * granules / splits);
  const int chunks = (g1 - g0 + 3) / 4;
  const uint32_t lds0 = (uint32_t)(uintptr_t)lds;

  const uint8_t* w_row[NW];
  const uint8_t* s_row[NW];
#pragma unroll
  for (int j = 0; j < NW; ++j) {
    const size_t row = (size_t)e * N + min(n0 + j * 16 + fr, N - 1);
    w_row[j] = W + row * (K / 2) + fc * 16;
    s_row[j] = WS + row * (K / 32);
  }

  for (int r0 = lo + (int)(blockIdx.z / splits) * kRows; r0 < hi; r0 += groups * kRows) {
    const int r1 = min(hi, r0 + kRows);
    const int active = (r1 - r0 + 15) >> 4;
    const uint16_t* a_row[kDma];
#pragma unroll
    for (int i = 0; i < kDma; ++i)
      a_row[i] = A + (size_t)act_row(src, k_top, tokens, min(r0 + i * kStreamWaves + wave, r1 - 1)) * K;
    // Row i*8 + wave of the stage; lane l writes piece l, i.e. logical piece
    // l ^ (row % 16).  Past K the last piece is read again (never used).
    auto stage_a = [&](int c) {
      const uint32_t base = lds0 + (c % kStreamDepth) * kStage;
#pragma unroll
      for (int i = 0; i < kDma; ++i) {
        const int row = i * kStreamWaves + wave;
        const int k = min((g0 + c * 4) * 128 + (lane ^ (row & 15)) * 8, K - 8);
        dma16(a_row[i] + k, base + row * 1024);
      }
    };
    struct Codes {
      u32x4 w[NW][4];
      uint32_t s[NW][4];
    };
    auto load_w = [&](Codes& b, int c) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int g = min(g0 + c * 4 + i, granules - 1);
#pragma unroll
        for (int j = 0; j < NW; ++j) {
          b.w[j][i] = ld16(w_row[j] + (size_t)g * 64);
          b.s[j][i] = *reinterpret_cast<const uint32_t*>(s_row[j] + (size_t)g * 4);
        }
      }
    };
    f32x4 acc[NMT][NW];
#pragma unroll
    for (int m = 0; m < NMT; ++m)
#pragma unroll
      for (int j = 0; j < NW; ++j) acc[m][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    auto compute = [&](const Codes& b, int c) {
      const uint8_t* st = lds + (c % kStreamDepth) * kStage;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (g0 + c * 4 + i < g1) {
          float scale[NW];
#pragma unroll
          for (int j = 0; j < NW; ++j)
            scale[j] = __uint_as_float(((b.s[j][i] >> (8 * fc)) & 0xffu) << 23);
#pragma unroll
          for (int s = 0; s < 4; ++s) {
            u32x4 wf[NW];
#pragma unroll
            for (int j = 0; j < NW; ++j) {
              const uint32_t c4 = b.w[j][i][s];
              wf[j][0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c4, scale[j], 0));
              wf[j][1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c4, scale[j], 1));
              wf[j][2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c4, scale[j], 2));
              wf[j][3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c4, scale[j], 3));
            }
#pragma unroll
            for (int m = 0; m < NMT; ++m) {
              if (m < active) {
                const u32x4 af = ld16(st + (m * 16 + fr) * 1024 + i * 256 + (((4 * fc + s) ^ fr) << 4));
#pragma unroll
                for (int j = 0; j < NW; ++j) acc[m][j] = mfma_bf16(wf[j], af, acc[m][j]);
              }
            }
          }
        }
      }
    };
    // Chunk c's activations are staged two chunks ahead, its codes one.
    Codes b0, b1;
    __syncthreads();                                 // the last row group's reads are done
    stage_a(0);
    if (chunks > 1) stage_a(1);
    load_w(b0, 0);
    auto step = [&](const Codes& now, Codes& next, int c) {
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // own DMA of chunk c (and older loads)
      __syncthreads();
      if (c + 2 < chunks) stage_a(c + 2);
      if (c + 1 < chunks) load_w(next, c + 1);
      compute(now, c);
    };
    for (int c = 0; c < chunks; c += 2) {
      step(b0, b1, c);
      if (c + 1 < chunks) step(b1, b0, c + 1);
    }

    // Lane: row m*16 + fr, columns n0 + j*16 + 4 fc .. + 3.
#pragma unroll
    for (int m = 0; m < NMT; ++m) {
      const int r = r0 + m * 16 + fr;
      if (m >= active || r >= r1) continue;
#pragma unroll
      for (int j = 0; j < NW; ++j) {
        const int n = n0 + j * 16 + 4 * fc;
        if (n >= N) continue;
        f32x4 v = acc[m][j];
        if (splits > 1) {
          *reinterpret_cast<f32x4*>(partial + ((size_t)split * rows_cap + r) * N + n) = v;
          continue;
        }
        if (bias) {
          const uint2 b = *reinterpret_cast<const uint2*>(bias + (size_t)e * N + n);
          v[0] += __uint_as_float(b.x << 16);
          v[1] += __uint_as_float(b.x & 0xffff0000u);
          v[2] += __uint_as_float(b.y << 16);
          v[3] += __uint_as_float(b.y & 0xffff0000u);
        }
        if constexpr (UP)
          *reinterpret_cast<uint2*>(static_cast<uint16_t*>(out) + (size_t)r * N + n) =
              make_uint2(pack_bf16x2(gelu_erf(v[0]), gelu_erf(v[1])),
                         pack_bf16x2(gelu_erf(v[2]), gelu_erf(v[3])));
        else
          *reinterpret_cast<f32x4*>(static_cast<float*>(out) + (size_t)r * N + n) = v;
      }
    }
  }
}

// The parts of k summed in order, then bias and GELU.  Block = rows blockIdx.y of the
// dispatch; its expert is found from the offsets.
template <bool UP>
__global__ __launch_bounds__(256) void mx_split_sum_kernel(
    const int32_t* __restrict__ offsets, int E, int rows_cap, const uint16_t* __restrict__ bias,
    void* __restrict__ out, int N, int splits, const float* __restrict__ partial) {
  const int r = blockIdx.y, n = (blockIdx.x * 256 + threadIdx.x) * 4;
  int e = 0;
  if (bias) {
    // The expert of row r: as many offsets [1, E] as are <= r lie before it.
    int before = 0;
    for (int i = threadIdx.x & 63; i < E; i += 64) before += offsets[i + 1] <= r;
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) before += __shfl_xor(before, o);
    e = min(before, E - 1);
  }
  if (n >= N || r < offsets[0] || r >= min(offsets[E], rows_cap)) return;
  f32x4 v = *reinterpret_cast<const f32x4*>(partial + (size_t)r * N + n);
  for (int s = 1; s < splits; ++s)
    v += *reinterpret_cast<const f32x4*>(partial + ((size_t)s * rows_cap + r) * N + n);
  if (bias) {
    const uint2 b = *reinterpret_cast<const uint2*>(bias + (size_t)e * N + n);
    v[0] += __uint_as_float(b.x << 16);
    v[1] += __uint_as_float(b.x & 0xffff0000u);
    v[2] += __uint_as_float(b.y << 16);
    v[3] += __uint_as_float(b.y & 0xffff0000u);
  }
  if constexpr (UP)
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(out) + (size_t)r * N + n) =
        make_uint2(pack_bf16x2(gelu_erf(v[0]), gelu_erf(v[1])), pack_bf16x2(gelu_erf(v[2]), gelu_erf(v[3])));
  else
    *reinterpret_cast<f32x4*>(static_cast<float*>(out) + (size_t)r * N + n) = v;
}

// Parts of k on the streaming path: enough blocks for two per CU from the experts
// that can have rows, at least 512 of k in each part, and only while the partial sums
// stay small beside the codes (at most 64 rows in all).
static int stream_splits(int T, int k, int E, int N, int K) {
  const long rows = (long)T * k;
  if (rows > 64) return 1;
  const long blocks = std::min<long>(E, rows) * ((N + kStreamCols - 1) / kStreamCols);
  return (int)std::max(1L, std::min({8L, K / 512L, 512 / blocks}));
}

size_t mx_partial_bytes(int T, int k, int E, int N, int K) {
  const int s = stream_splits(T, k, E, N, K);
  return s > 1 ? (size_t)s * T * k * N * 4 : 0;
}

// Experts averaging at least 48 rows run the LDS-tiled kernel, the rest stream.  The tiled
// kernel's loads run up to two steps of 256 k ahead, so it starts at k = 512.
static bool tiled(int T, int k, int E, int K) { return (long)T * k >= 48L * E && K >= 512; }

size_t mx_act_bytes(int T, int k, int E, int N, int K, bool fp4) {
  const long rows = (long)T * k;
  return tiled(T, k, E, K) ? mx_tile_bytes(rows, E, N, K, fp4) : fp4 ? (size_t)rows * K * 2 : 0;
}

template <bool UP, int NMT>
static void launch_stream(const MxFfnArgs& a, const void* act, int splits, hipStream_t s) {
  const int R = a.T * a.k;
  // Row groups in flight: the average expert's; fuller experts loop.
  const int groups = std::max(1, std::min((a.T + 16 * NMT - 1) / (16 * NMT),
                                          (R / a.E + 16 * NMT - 1) / (16 * NMT)));
  const dim3 grid((a.N + kStreamCols - 1) / kStreamCols, a.E, groups * splits);
  mx_stream_kernel<UP, NMT><<<grid, 512, 0, s>>>(
      static_cast<const uint16_t*>(act), a.src, a.k, a.T, a.offsets, R, a.w, a.ws,
      static_cast<const uint16_t*>(a.bias), a.out, a.N, a.K, splits, a.partial);
  if (splits > 1)
    mx_split_sum_kernel<UP><<<dim3((a.N / 4 + 255) / 256, R), 256, 0, s>>>(
        a.offsets, a.E, R, static_cast<const uint16_t*>(a.bias), a.out, a.N, splits, a.partial);
}

hipError_t launch_mx_ffn(const MxFfnArgs& a, hipStream_t s) {
  if (tiled(a.T, a.k, a.E, a.K)) return launch_mx_tile(a, s);
  const void* act = a.a;
  if (a.fp4) {
    // The values the 4-bit activations stand for, as bf16: exact in the products.
    if (hipError_t e = launch_mx_requantize(a.a, a.a_rows, a.K, a.act, s)) return e;
    act = a.act;
  }
  const int splits = stream_splits(a.T, a.k, a.E, a.N, a.K);
  const bool one = a.T <= 16;                       // no expert holds more than 16 rows
  if (a.up)
    one ? launch_stream<true, 1>(a, act, splits, s) : launch_stream<true, 2>(a, act, splits, s);
  else
    one ? launch_stream<false, 1>(a, act, splits, s) : launch_stream<false, 2>(a, act, splits, s);
  return hipGetLastError();
}

}  // namespace moe
