// A projection shared by all tokens, with a low-rank adapter of each token's own beside it:
//   y_t = act(W x_t + bias + scale_a B_a (A_a x_t)),  a = adapter[t]; outside [0, N): no adapter
//
// Two kernels: u_t = scale_a A_a x_t, then the projection, which adds B_a u_t at its end.
// The tokens stay in their order.  A tile of tokens runs once through the list of the
// different adapters that its tokens have: one for a long request, as many as tokens in a decode batch.
#include <algorithm>
#include <type_traits>

#include "device_common.h"
#include "lora.h"

namespace moe {

constexpr int kWaves = 8;              // of a block, k steps dealt in turn

// Rows of `mask` (a bit per lane) one group of equal ids at a time: f(id, lanes that have it,
// index of the group).  Uniform over the wave.
template <typename F>
__device__ __forceinline__ void for_ids(int id, uint64_t mask, F f) {
  for (int i = 0; mask; ++i) {
    const int one = __builtin_amdgcn_readlane(id, __ffsll((unsigned long long)mask) - 1);
    const uint64_t same = __ballot(id == one) & mask;
    f(one, same, i);
    mask &= ~same;
  }
}

// Fragments of `NA` and `NB` 16-row groups, 32 values of k each, through U register stages; the
// waves of a block take every kWaves-th step of k.  acc[j][m] += A_j B_m^T.
template <int NA, int NB, int U>
__device__ __forceinline__ void dot_rows(const uint16_t* (&pa)[NA], const uint16_t* (&pb)[NB], int steps, int wave,
                                         f32x4 (&acc)[NA][NB]) {
  u32x4 fa[U][NA], fb[U][NB];
  const int mine = (steps - wave + kWaves - 1) / kWaves, last = steps - 1;
  auto load = [&](int slot, int i) {                 // past the end: the last step again, not used
    const int k = min(wave + i * kWaves, last) * 32;
#pragma unroll
    for (int j = 0; j < NA; ++j) fa[slot][j] = ld16(pa[j] + k);
#pragma unroll
    for (int m = 0; m < NB; ++m) fb[slot][m] = ld16(pb[m] + k);
  };
  auto multiply = [&](int slot) {
#pragma unroll
    for (int j = 0; j < NA; ++j)
#pragma unroll
      for (int m = 0; m < NB; ++m) acc[j][m] = mfma_bf16(fa[slot][j], fb[slot][m], acc[j][m]);
  };
#pragma unroll
  for (int q = 0; q < U; ++q) load(q, q);
  int i = 0;
  for (; i + U <= mine; i += U) {
#pragma unroll
    for (int q = 0; q < U; ++q) {
      multiply(q);
      load(q, i + U + q);
    }
  }
#pragma unroll
  for (int q = 0; q < U; ++q)
    if (i + q < mine) multiply(q);
}

// ---------------------------------------------------------------------------
// u: a block has 16 MT tokens and, of the groups (adapter, 64 ranks) that they need, every
// gridDim.y-th.  Its waves share out k, so the sums meet in LDS.  Bound by reading x, with few
// tokens by reading A.
// ---------------------------------------------------------------------------
struct ShrinkArgs {
  LoraArgs a;
  bool terms;                          // bf16 terms, else fp32
};

template <int MT, int RT>
__global__ __launch_bounds__(kWaves * 64) void lora_shrink_kernel(ShrinkArgs p) {
  constexpr int kRows = 16 * MT, kRanks = 16 * RT;
  __shared__ __attribute__((aligned(16))) float part[kWaves][kRows][kRanks];
  const LoraArgs& a = p.a;
  const int T = a.sh.T, d = a.sh.d, rank = a.sh.rank, pitch = (rank + 15) / 16 * 16;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int fr = lane & 15, fc = lane >> 4, t0 = blockIdx.x * kRows;
  const int own = t0 + lane < T && lane < kRows ? a.adapter[t0 + lane] : -1;   // lane l: token t0 + l
  const uint16_t* px[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) px[m] = a.x + (size_t)min(t0 + m * 16 + fr, T - 1) * d + fc * 8;
  const int chunks = (pitch + kRanks - 1) / kRanks;
  for_ids(own, __ballot((uint32_t)own < (uint32_t)a.sh.N), [&](int id, uint64_t, int i) {
    for (int c = 0; c < chunks; ++c) {
      if ((uint32_t)(i * chunks + c) % gridDim.y != blockIdx.y) continue;
      const int r0 = c * kRanks;
      const uint16_t* pa[RT];
#pragma unroll
      for (int j = 0; j < RT; ++j)
        pa[j] = a.a + ((size_t)id * rank + min(r0 + j * 16 + fr, rank - 1)) * d + fc * 8;
      f32x4 acc[RT][MT] = {};
      dot_rows<RT, MT, (MT + RT >= 6 ? 2 : 4)>(pa, px, d / 32, wave, acc);
      // A lane has ranks 4 fc .. + 3 of token fr.
#pragma unroll
      for (int j = 0; j < RT; ++j)
#pragma unroll
        for (int m = 0; m < MT; ++m)
          *reinterpret_cast<f32x4*>(&part[wave][m * 16 + fr][j * 16 + fc * 4]) = acc[j][m];
      __syncthreads();
      const float scale = a.scale ? a.scale[id] : 1.f;
      for (int o = threadIdx.x; o < kRows * kRanks / 2; o += kWaves * 64) {   // two ranks a thread
        const int row = o / (kRanks / 2), r = o % (kRanks / 2) * 2;
        float v[2] = {0.f, 0.f};
#pragma unroll
        for (int w = 0; w < kWaves; ++w) v[0] += part[w][row][r], v[1] += part[w][row][r + 1];
        const int t = t0 + row;
        if (t >= T || r0 + r >= pitch || a.adapter[t] != id) continue;
#pragma unroll
        for (int q = 0; q < 2; ++q) v[q] = r0 + r + q < rank ? v[q] * scale : 0.f;
        const size_t at = (size_t)t * pitch + r0 + r;
        if (!p.terms) {
          *reinterpret_cast<float2*>(static_cast<float*>(a.u) + at) = make_float2(v[0], v[1]);
        } else {
          uint16_t* u = static_cast<uint16_t*>(a.u);
          const int terms = a.sh.f32_out ? 3 : 2;
          for (int q = 0; q < terms; ++q) {
            const uint32_t h = pack_bf16x2(v[0], v[1]);
            *reinterpret_cast<uint32_t*>(u + (size_t)q * T * pitch + at) = h;
            // what the term left over; nothing of an infinity
            v[0] = (h & 0x7f80u) == 0x7f80u ? 0.f : v[0] - __uint_as_float(h << 16);
            v[1] = (h & 0x7f800000u) == 0x7f800000u ? 0.f : v[1] - __uint_as_float(h & 0xffff0000u);
          }
        }
      }
      __syncthreads();
    }
  });
}

// ---------------------------------------------------------------------------
// The projection with few tokens, bound by the bytes of W: a block has 16 NMT tokens and 16 NNT
// columns, its waves share out k, fragments go straight from memory to registers.  The sums meet
// in LDS, where a thread finishes an output: bias, B_a u, activation.
// ---------------------------------------------------------------------------
template <int NMT, int NNT>
__global__ __launch_bounds__(kWaves * 64) void lora_stream_kernel(LoraArgs a) {
  constexpr int kRows = 16 * NMT, kCols = 16 * NNT;
  __shared__ __attribute__((aligned(16))) float part[kWaves][kRows][kCols];
  const int T = a.sh.T, d = a.sh.d, n = a.sh.n, rank = a.sh.rank, pitch = (rank + 15) / 16 * 16;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int fr = lane & 15, fc = lane >> 4, t0 = blockIdx.y * kRows, n0 = blockIdx.x * kCols;
  const uint16_t *px[NMT], *pw[NNT];
#pragma unroll
  for (int m = 0; m < NMT; ++m) px[m] = a.x + (size_t)min(t0 + m * 16 + fr, T - 1) * d + fc * 8;
#pragma unroll
  for (int j = 0; j < NNT; ++j) pw[j] = a.w + (size_t)min(n0 + j * 16 + fr, n - 1) * d + fc * 8;
  f32x4 acc[NNT][NMT] = {};
  dot_rows<NNT, NMT, (NMT + NNT >= 8 ? 2 : NMT + NNT >= 5 ? 4 : 8)>(pw, px, d / 32, wave, acc);
#pragma unroll
  for (int j = 0; j < NNT; ++j)
#pragma unroll
    for (int m = 0; m < NMT; ++m)
      *reinterpret_cast<f32x4*>(&part[wave][m * 16 + fr][j * 16 + fc * 4]) = acc[j][m];
  __syncthreads();
  for (int o = threadIdx.x; o < kRows * kCols; o += kWaves * 64) {
    const int row = o / kCols, col = o % kCols, t = t0 + row, c = n0 + col;
    if (t >= T || c >= n) continue;
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) v += part[w][row][col];
    if (a.bias) v += bf16_to_f32(a.bias[c]);
    const int id = a.adapter[t];
    if ((uint32_t)id < (uint32_t)a.sh.N) {
      const uint16_t* b = a.b + ((size_t)id * n + c) * rank;
      const float* u = static_cast<const float*>(a.u) + (size_t)t * pitch;
      float s = 0.f;
      for (int r = 0; r < rank; r += 8) {
        const u32x4 q = ld16(b + r);
        const f32x4 u0 = *reinterpret_cast<const f32x4*>(u + r), u1 = *reinterpret_cast<const f32x4*>(u + r + 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float x0 = i < 2 ? u0[2 * i] : u1[2 * i - 4], x1 = i < 2 ? u0[2 * i + 1] : u1[2 * i - 3];
          s = fmaf(__uint_as_float(q[i] << 16), x0, s);
          s = fmaf(__uint_as_float(q[i] & 0xffff0000u), x1, s);
        }
      }
      v += s;
    }
    if (a.sh.f32_out) {
      static_cast<float*>(a.y)[(size_t)t * n + c] = a.sh.gelu ? gelu_erf(v) : v;
    } else {
      static_cast<uint16_t*>(a.y)[(size_t)t * n + c] = (uint16_t)pack_bf16x2(a.sh.gelu ? gelu_for_bf16(v) : v, 0.f);
    }
  }
}

// ---- launches ------------------------------------------------------------------------------
size_t lora_u_bytes(const LoraShape& s) {
  return (size_t)s.T * lora_pitch(s.rank) * (lora_tiled(s) ? 2 * lora_terms(s) : 4);
}

template <int MT>
static void run_shrink(const ShrinkArgs& p, hipStream_t s) {
  const LoraShape& h = p.a.sh;
  const int tiles = (h.T + 16 * MT - 1) / (16 * MT), pitch = lora_pitch(h.rank);
  const int groups = std::min(h.N, 16 * MT) * ((pitch + 63) / 64);
  // Few tiles: a block for every group that a tile can have.
  const dim3 grid(tiles, tiles >= 256 ? 1 : std::min(groups, std::max(1, 512 / tiles)));
  if (pitch <= 16) lora_shrink_kernel<MT, 1><<<grid, kWaves * 64, 0, s>>>(p);
  else if (pitch <= 32) lora_shrink_kernel<MT, 2><<<grid, kWaves * 64, 0, s>>>(p);
  else lora_shrink_kernel<MT, 4><<<grid, kWaves * 64, 0, s>>>(p);
}

hipError_t launch_lora(const LoraArgs& a, hipStream_t s) {
  const bool tiled = lora_tiled(a.sh);
  const ShrinkArgs p{a, tiled};
  if (a.sh.T >= 16384) run_shrink<4>(p, s);
  else if (a.sh.T >= 8192) run_shrink<2>(p, s);
  else run_shrink<1>(p, s);
  if (hipError_t e = hipGetLastError()) return e;
  if (tiled) return launch_lora_tile(a, s);
  auto run = [&](auto mt, auto nt) {
    constexpr int M = decltype(mt)::value, C = decltype(nt)::value;
    const dim3 grid((a.sh.n + 16 * C - 1) / (16 * C), (a.sh.T + 16 * M - 1) / (16 * M));
    lora_stream_kernel<M, C><<<grid, kWaves * 64, 0, s>>>(a);
  };
  using std::integral_constant;
  const integral_constant<int, 1> one;
  const integral_constant<int, 2> two;
  const integral_constant<int, 4> four;
  if (a.sh.T <= 16) run(one, one);
  else if (a.sh.T <= 32) a.sh.n >= 8192 ? run(two, two) : run(two, one);
  else if ((long)((a.sh.T + 63) / 64) * a.sh.n >= 64 * 256) run(four, four);
  else run(four, one);
  return hipGetLastError();
}

}  // namespace moe
