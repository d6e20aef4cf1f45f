// A projection shared by all tokens, with a low-rank adapter of each token's own beside it:
//   y_t = act(W x_t + bias + scale_a B_a (A_a x_t)),  a = adapter[t]; outside [0, N): no adapter
//
// Two kernels: u_t = scale_a A_a x_t, then the projection, which adds B_a u_t at its end.
// The tokens stay in their order.  A tile of tokens runs once through the list of the
// different adapters that its tokens have: one for a long request, as many as tokens in a
// decode batch.
#include <algorithm>
#include <type_traits>

#include "device_common.h"
#include "lora.h"

namespace moe {

// Fragments of `NA` and `NB` 16-row groups, 32 values of k each, through U register stages; the
// WAVES waves of a block take every WAVES-th step of k.  acc[j][m] += A_j B_m^T.
template <int NA, int NB, int U, int WAVES>
__device__ __forceinline__ void dot_rows(const uint16_t* (&pa)[NA], const uint16_t* (&pb)[NB], int steps, int wave,
                                         f32x4 (&acc)[NA][NB]) {
  u32x4 fa[U][NA], fb[U][NB];
  const int mine = (steps - wave + WAVES - 1) / WAVES, last = steps - 1;
  auto load = [&](int slot, int i) {                 // past the end: the last step again, not used
    const int k = min(wave + i * WAVES, last) * 32;
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
// u: a block has 16 MT tokens and first lists the different adapters among them.  An adapter is
// pitch / 16 groups of 16 ranks; a pass over k takes NS groups, of one adapter or of several, so
// that x is read once for a few adapters; block y takes every gridDim.y-th pass.  The
// waves share out k, so the sums meet in LDS.  Bound by reading x, with few tokens by
// the latency of reading A.
// ---------------------------------------------------------------------------
struct ShrinkArgs {
  LoraArgs a;
  bool terms;                          // bf16 terms, else fp32
};

template <int MT, int NS, int WAVES>
__global__ __launch_bounds__(WAVES * 64) void lora_shrink_kernel(ShrinkArgs p) {
  constexpr int kRows = 16 * MT, kRanks = 16 * NS;
  __shared__ __attribute__((aligned(16))) float part[WAVES][kRows][kRanks];
  __shared__ int list[kRows];
  const LoraArgs& a = p.a;
  const int T = a.sh.T, d = a.sh.d, rank = a.sh.rank, pitch = (rank + 15) / 16 * 16, per = pitch / 16;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int fr = lane & 15, fc = lane >> 4, t0 = blockIdx.x * kRows;
  const int own = t0 + lane < T && lane < kRows ? a.adapter[t0 + lane] : -1;   // lane l: token t0 + l
  int count = 0;
  for (uint64_t left = __ballot((uint32_t)own < (uint32_t)a.sh.N); left; ++count) {
    const int id = __builtin_amdgcn_readlane(own, __ffsll((unsigned long long)left) - 1);
    left &= ~__ballot(own == id);
    if (threadIdx.x == 0) list[count] = id;
  }
  __syncthreads();
  const uint16_t* px[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) px[m] = a.x + (size_t)min(t0 + m * 16 + fr, T - 1) * d + fc * 8;
  const int groups = count * per;
  for (int g0 = blockIdx.y * NS; g0 < groups; g0 += gridDim.y * NS) {
    const uint16_t* pa[NS];
#pragma unroll
    for (int j = 0; j < NS; ++j) {
      const int g = min(g0 + j, groups - 1);
      pa[j] = a.a + ((size_t)list[g / per] * rank + min(g % per * 16 + fr, rank - 1)) * d + fc * 8;
    }
    f32x4 acc[NS][MT] = {};
    dot_rows<NS, MT, (NS + MT >= 8 ? 2 : NS + MT >= 4 ? 4 : 8), WAVES>(pa, px, d / 32, wave, acc);
    // A lane has ranks 4 fc .. + 3 of token fr.
#pragma unroll
    for (int j = 0; j < NS; ++j)
#pragma unroll
      for (int m = 0; m < MT; ++m)
        *reinterpret_cast<f32x4*>(&part[wave][m * 16 + fr][j * 16 + fc * 4]) = acc[j][m];
    __syncthreads();
    for (int o = threadIdx.x; o < kRows * kRanks / 2; o += WAVES * 64) {   // two ranks a thread
      const int row = o / (kRanks / 2), r = o % (kRanks / 2) * 2, g = g0 + r / 16, t = t0 + row;
      if (t >= T || g >= groups) continue;
      const int id = list[g / per], at_rank = g % per * 16 + r % 16;
      if (a.adapter[t] != id) continue;
      float v[2] = {0.f, 0.f};
#pragma unroll
      for (int w = 0; w < WAVES; ++w) v[0] += part[w][row][r], v[1] += part[w][row][r + 1];
      const float scale = a.scale ? a.scale[id] : 1.f;
#pragma unroll
      for (int q = 0; q < 2; ++q) v[q] = at_rank + q < rank ? v[q] * scale : 0.f;
      const size_t at = (size_t)t * pitch + at_rank;
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
}

// ---------------------------------------------------------------------------
// The projection with few tokens, bound by the bytes of W: a block has 16 NMT tokens and 16 NNT
// columns, its eight waves share out k, fragments go straight from memory to registers.  The
// sums meet in LDS, where a thread finishes an output: bias, B_a u, activation.
// FUSED > 0, one token: its adapter's 16 FUSED ranks are further rows beside the block's columns of
// W, so every block has u itself and there is one launch; its reads of A come from L2.
// ---------------------------------------------------------------------------
constexpr int kWaves = 8;

// Eight ranks of B times eight values of u.
__device__ __forceinline__ float dot8(const u32x4& q, const float* u, float s) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    s = fmaf(__uint_as_float(q[i] << 16), u[2 * i], s);
    s = fmaf(__uint_as_float(q[i] & 0xffff0000u), u[2 * i + 1], s);
  }
  return s;
}

template <int NMT, int NNT, int FUSED>
__global__ __launch_bounds__(kWaves * 64) void lora_stream_kernel(LoraArgs a) {
  static_assert(!FUSED || NMT == 1, "one token");
  constexpr int kRows = 16 * NMT, kCols = 16 * NNT, kAll = kCols + 16 * FUSED, NA = NNT + FUSED;
  constexpr int kThreads = kWaves * 64, kOut = (kRows * kCols + kThreads - 1) / kThreads;
  constexpr bool kEarly = kOut <= 2;                 // the first 16 ranks of B and u: loaded before the sums meet
  __shared__ __attribute__((aligned(16))) float part[kWaves][kRows][kAll];
  __shared__ __attribute__((aligned(16))) float su[FUSED ? 16 * FUSED : 4];
  __shared__ int ids[kRows];
  const int T = a.sh.T, d = a.sh.d, n = a.sh.n, rank = a.sh.rank, pitch = (rank + 15) / 16 * 16;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int fr = lane & 15, fc = lane >> 4, t0 = blockIdx.y * kRows, n0 = blockIdx.x * kCols;
  if (threadIdx.x < kRows) {
    const int id = t0 + (int)threadIdx.x < T ? a.adapter[t0 + threadIdx.x] : -1;
    ids[threadIdx.x] = (uint32_t)id < (uint32_t)a.sh.N ? id : -1;
  }
  const uint16_t *px[NMT], *pw[NA];
#pragma unroll
  for (int m = 0; m < NMT; ++m) px[m] = a.x + (size_t)min(t0 + m * 16 + fr, T - 1) * d + fc * 8;
#pragma unroll
  for (int j = 0; j < NNT; ++j) pw[j] = a.w + (size_t)min(n0 + j * 16 + fr, n - 1) * d + fc * 8;
  __syncthreads();
#pragma unroll
  for (int j = 0; j < FUSED; ++j)                    // no adapter: any will do, it is not used
    pw[NNT + j] = a.a + ((size_t)max(ids[0], 0) * rank + min(j * 16 + fr, rank - 1)) * d + fc * 8;
  f32x4 acc[NA][NMT] = {};
  dot_rows<NA, NMT, (NMT + NA >= 7 ? 2 : NMT + NA >= 4 ? 4 : 8), kWaves>(pw, px, d / 32, wave, acc);

  // Output i of a thread, columns fastest.
  auto where = [&](int i, int& t, int& c, int& id) {
    const int o = i * kThreads + threadIdx.x;
    t = t0 + o / kCols;
    c = n0 + o % kCols;
    const bool in = o < kRows * kCols && t < T && c < n;
    id = in ? ids[o / kCols] : -1;
    return in;
  };
  u32x4 qb[kEarly ? kOut : 1][2];
  f32x4 qu[kEarly && !FUSED ? kOut : 1][4];
  if constexpr (kEarly) {
#pragma unroll
    for (int i = 0; i < kOut; ++i) {
      int t, c, id;
      where(i, t, c, id);
      if (id < 0) continue;
      const uint16_t* b = a.b + ((size_t)id * n + c) * rank;
      qb[i][0] = ld16(b);
      qb[i][1] = rank > 8 ? ld16(b + 8) : u32x4{0, 0, 0, 0};
      if constexpr (!FUSED) {
        const float* u = static_cast<const float*>(a.u) + (size_t)t * pitch;
#pragma unroll
        for (int q = 0; q < 4; ++q) qu[i][q] = *reinterpret_cast<const f32x4*>(u + 4 * q);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < NA; ++j)
#pragma unroll
    for (int m = 0; m < NMT; ++m)
      *reinterpret_cast<f32x4*>(&part[wave][m * 16 + fr][j * 16 + fc * 4]) = acc[j][m];
  __syncthreads();
  if constexpr (FUSED > 0) {
    if (threadIdx.x < 16 * FUSED) {
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) v += part[w][0][kCols + threadIdx.x];
      su[threadIdx.x] = (int)threadIdx.x < rank ? v * (a.scale && ids[0] >= 0 ? a.scale[ids[0]] : 1.f) : 0.f;
    }
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < kOut; ++i) {
    int t, c, id;
    if (!where(i, t, c, id)) continue;
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) v += part[w][t - t0][c - n0];
    if (a.bias) v += bf16_to_f32(a.bias[c]);
    if (id >= 0) {
      const uint16_t* b = a.b + ((size_t)id * n + c) * rank;
      const float* u = FUSED ? su : static_cast<const float*>(a.u) + (size_t)t * pitch;
      float s = 0.f;
      int r = 0;
      if constexpr (kEarly) {
        const float* u0 = FUSED ? su : reinterpret_cast<const float*>(qu[FUSED ? 0 : i]);
        s = dot8(qb[i][0], u0, s);
        if (rank > 8) s = dot8(qb[i][1], u0 + 8, s);
        r = 16;
      }
      for (; r < rank; r += 8) {
        f32x4 v4[2] = {*reinterpret_cast<const f32x4*>(u + r), *reinterpret_cast<const f32x4*>(u + r + 4)};
        s = dot8(ld16(b + r), reinterpret_cast<const float*>(v4), s);
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

template <int MT, int NS, int WAVES>
static void run_shrink(const ShrinkArgs& p, int passes, hipStream_t s) {
  const dim3 grid((p.a.sh.T + 16 * MT - 1) / (16 * MT), passes);
  lora_shrink_kernel<MT, NS, WAVES><<<grid, WAVES * 64, 0, s>>>(p);
}

static void launch_shrink(const ShrinkArgs& p, hipStream_t s) {
  const LoraShape& h = p.a.sh;
  const int per = lora_pitch(h.rank) / 16;
  const int tiles = (h.T + 15) / 16, most = std::min(h.N, 16) * per;   // groups that a tile of 16 can have
  if (tiles <= 64) run_shrink<1, 1, 16>(p, std::min(most, 1024 / tiles), s);
  else if (tiles <= 256) run_shrink<1, 4, 8>(p, std::max(1, std::min((most + 3) / 4, 512 / tiles)), s);
  else if (tiles <= 1024) run_shrink<2, 4, 8>(p, 1, s);
  else run_shrink<4, 4, 8>(p, 1, s);
}

hipError_t launch_lora(const LoraArgs& a, hipStream_t s) {
  using std::integral_constant;
  const integral_constant<int, 0> none;
  const integral_constant<int, 1> one;
  const integral_constant<int, 2> two;
  const integral_constant<int, 4> four;
  auto stream = [&](auto mt, auto nt, auto fused) {
    constexpr int M = decltype(mt)::value, C = decltype(nt)::value;
    const dim3 grid((a.sh.n + 16 * C - 1) / (16 * C), (a.sh.T + 16 * M - 1) / (16 * M));
    lora_stream_kernel<M, C, decltype(fused)::value><<<grid, kWaves * 64, 0, s>>>(a);
    return hipGetLastError();
  };
  if (a.sh.T == 1 && a.sh.rank <= 32) {
    auto wide = [&](auto fused) {
      return a.sh.n >= 12288 ? stream(one, four, fused) : a.sh.n >= 8192 ? stream(one, two, fused) : stream(one, one, fused);
    };
    return a.sh.rank <= 16 ? wide(one) : wide(two);
  }
  const bool tiled = lora_tiled(a.sh);
  launch_shrink(ShrinkArgs{a, tiled}, s);
  if (hipError_t e = hipGetLastError()) return e;
  if (tiled) return launch_lora_tile(a, s);
  if (a.sh.T <= 16) return a.sh.n >= 8192 ? stream(one, two, none) : stream(one, one, none);
  if (a.sh.T <= 32) return a.sh.n >= 8192 ? stream(two, two, none) : stream(two, one, none);
  if ((long)((a.sh.T + 63) / 64) * a.sh.n >= 64 * 256) return stream(four, four, none);
  return stream(four, one, none);
}

}  // namespace moe
