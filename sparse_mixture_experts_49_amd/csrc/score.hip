// The scored router on gfx950: logits on MFMA, then scores, groups, top-k and
// weights, one wave per token, and the sums over tokens that the losses need.
//
// Web page "Mixture of Experts: Scaling Parameters Without Scaling Compute",
// sections "The MoE layer" (router, top-k, renormalisation) and "The central
// problem: load balancing" (balance loss, z-loss, selection-only bias), with
// sigmoid scores and group-limited selection added.
#include <algorithm>
#include <type_traits>

#include "device_common.h"
#include "score.h"

namespace moe {

// Many tokens: the LDS-tiled kernel, few: the direct one.  Whole calls, direct and tiled: d =
// 4096, 256 experts, 512 tokens 30 and 32 us, 1024 tokens 46 and 30; d = 2048, 64 experts,
// 1024 tokens 17.5 and 17.7 us, 2048 tokens 22 and 18.
static bool score_tiled(const ScoreShape& s) { return s.T >= (s.E <= 64 ? 1536 : 768); }

int score_parts(const ScoreShape& s) {
  if (score_tiled(s)) {
    // One part where the tiles fill more than half the chip; else enough to fill it, two
    // steps or more in each.
    const long tiles = (s.T + 63) / 64, steps = s.d / (s.bf16 ? 64 : 32);
    return tiles > 128 ? 1 : (int)std::max(1L, std::min(256 / tiles, steps / 2));
  }
  // Enough waves to cover the chip twice (512 blocks), no part under 128 of d.
  const long blocks = (long)((s.T + 15) / 16) * ((s.E + 63) / 64);
  const long most = std::min(32L, s.d / 128L);
  return (int)std::max(1L, std::min(most, 512 / blocks));
}

// Partial logits: wave w of block (t-tile, e-tile, part) multiplies 16 tokens by
// 16 experts over its part of d, operands straight from memory to registers.  Few tokens:
// bound by latency, so d is split until the chip has work (1 token, d = 2048, 64 experts 3.0 us).
template <typename T>
__global__ __launch_bounds__(256) void score_logits_kernel(const T* __restrict__ x,
                                                           const T* __restrict__ w, int tokens,
                                                           int d, int E, int parts,
                                                           float* __restrict__ part,
                                                           uint32_t* __restrict__ done) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int fr = lane & 15, fc = lane >> 4;
  const int t0 = blockIdx.x * 16, e0 = blockIdx.y * 64 + wave * 16, p = blockIdx.z;
  if (t0 == 0 && e0 == 0 && p == 0 && lane == 0) *done = 0u;   // score_reduce_kernel's counter
  if (e0 >= E) return;
  const int chunks = d / 128;
  const int c0 = (int)((long)p * chunks / parts), c1 = (int)((long)(p + 1) * chunks / parts);
  const T* xr = x + (size_t)min(t0 + fr, tokens - 1) * d;
  const T* wr = w + (size_t)min(e0 + fr, E - 1) * d;
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  for (int c = c0; c < c1; ++c) {
    if constexpr (sizeof(T) == 2) {
      u32x4 a[4], b[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        a[i] = ld16(xr + c * 128 + i * 32 + fc * 8);
        b[i] = ld16(wr + c * 128 + i * 32 + fc * 8);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) acc = mfma_bf16(a[i], b[i], acc);
    } else {
      f32x4 a[8], b[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        a[i] = *reinterpret_cast<const f32x4*>(xr + c * 128 + i * 16 + fc * 4);
        b[i] = *reinterpret_cast<const f32x4*>(wr + c * 128 + i * 16 + fc * 4);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) acc = mfma_f32(a[i][q], b[i][q], acc);
    }
  }
  // Lane: expert e0 + fr, tokens t0 + 4 fc + i.
  if (e0 + fr >= E) return;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int t = t0 + 4 * fc + i;
    if (t < tokens) part[((size_t)p * tokens + t) * E + e0 + fr] = acc[i];
  }
}

// Order-preserving integer of a selection value: larger = better, 1 = NaN, 0 is
// left for "not available".  -0 counts as +0.
__device__ __forceinline__ uint32_t order_key(float v) {
  if (v != v) return 1u;
  const uint32_t b = __float_as_uint(v == 0.f ? 0.f : v);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

// One value per lane's pair step of a reduction over 2^shift neighbouring lanes, o = 1, 2, 4,
// ...: permutations of quads, eights and rows of 16 (equal within the smaller groups by
// then, so a mirror pairs as an exchange would), beyond that a shuffle.
template <int STEP>
__device__ __forceinline__ float pair_of(float v) {
  const int i = (int)__float_as_uint(v);
  if constexpr (STEP == 0) return __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, i, 0xB1, 0xF, 0xF, false));
  if constexpr (STEP == 1) return __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, i, 0x4E, 0xF, 0xF, false));
  if constexpr (STEP == 2) return __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, i, 0x141, 0xF, 0xF, false));
  if constexpr (STEP == 3) return __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, i, 0x140, 0xF, 0xF, false));
  return __shfl_xor(v, 1 << STEP);
}

// What a wave needs to finish tokens: lane l holds experts l, l + 64, ... (PER of them).
// Straight-line code: lanes past E carry logit -inf and key 0 (one token per wave is bound by
// instruction issue and latency, branches cost most of both).  16384 tokens, 256 experts in 8
// groups, k = 8, with the sums: 28 us (17 MB of logits would take 4); one token 4.5 us.
template <int PER, bool TRAIN>
struct Finisher {
  int shift, gs;                 // lanes per group 2^shift, experts per group
  int gbit[PER];                 // lane that knows whether the group of expert j * 64 + l stays
  bool live[PER];                // j * 64 + l < E
  float bsel[PER];
  double pq[PER], pz;            // TRAIN: this wave's sums over its tokens
  int pl[PER];

  __device__ __forceinline__ void init(const ScoreArgs& a) {
    const int lane = __lane_id(), E = a.sh.E, G = a.groups;
    gs = E / G;
    shift = 0;
    while ((G << (shift + 1)) <= 64) ++shift;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const int e = j * 64 + lane;
      live[j] = e < E;
      gbit[j] = live[j] ? (e / gs) << shift : 0;
      bsel[j] = (a.b_select && live[j]) ? a.b_select[e] : 0.f;
      pq[j] = 0.0;
      pl[j] = 0;
    }
    pz = 0.0;
  }

  // One token from its logits (lanes past E: -inf); sel: 64 * PER floats of LDS of this wave.
  __device__ __forceinline__ void token(const ScoreArgs& a, int t, const float (&l)[PER], float* sel) {
    const int lane = __lane_id(), k = a.sh.k, G = a.groups;
    float s[PER];
    if ((TRAIN && a.z_loss) || !a.sigmoid) {
      float m = l[0], tot = 0.f;
#pragma unroll
      for (int j = 1; j < PER; ++j) m = fmaxf(m, l[j]);
      m = wave_max_f(m);
      m = m == -INFINITY ? 0.f : m;                // every logit -inf: all scores 0
#pragma unroll
      for (int j = 0; j < PER; ++j) tot += s[j] = exp_f32(l[j] - m);
      tot = wave_sum_f(tot);
      if (TRAIN && a.z_loss) {
        const double lse = (double)m + (double)__builtin_amdgcn_logf(tot) * 0.69314718055994530942;
        pz += lse * lse;
      }
      const float r = tot > 0.f ? 1.f / tot : tot != tot ? tot : 0.f;
#pragma unroll
      for (int j = 0; j < PER; ++j) s[j] *= r;
    }
    if (a.sigmoid) {
#pragma unroll
      for (int j = 0; j < PER; ++j) s[j] = sigmoid_f32(l[j]);
    }
    if (TRAIN) {
      float r = 1.f;
      if (a.sigmoid) {
        float q = 0.f;
#pragma unroll
        for (int j = 0; j < PER; ++j) q += s[j];
        q = wave_sum_f(q);
        r = 1.f / (q < kLeastSum ? kLeastSum : q);   // every score underflowed: q = 0
      }
#pragma unroll
      for (int j = 0; j < PER; ++j) pq[j] += (double)(s[j] * r);
    }

    uint32_t key[PER];
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const float v = s[j] + bsel[j];
      key[j] = live[j] ? order_key(v) : 0u;
      if (G > 1) sel[j * 64 + lane] = v == v ? v : -INFINITY;
    }
    if (G > 1) {
      // Lanes [g P, (g + 1) P), P = 2^shift, find the best two of group g.
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
      __builtin_amdgcn_wave_barrier();
      const int g = lane >> shift, P = 1 << shift, p = lane & (P - 1);
      const float* mine = sel + min(g, G - 1) * gs;
      float b0 = -INFINITY, b1 = -INFINITY;
      for (int i = 0; i < gs; i += 4 * P) {
        float v[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) v[q] = mine[min(i + q * P + p, gs - 1)];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          v[q] = i + q * P + p < gs ? v[q] : -INFINITY;
          b1 = fmaxf(b1, fminf(b0, v[q]));
          b0 = fmaxf(b0, v[q]);
        }
      }
      __builtin_amdgcn_wave_barrier();
      auto merge = [&](auto step) {
        constexpr int ST = decltype(step)::value;
        if (shift > ST) {
          const float c0 = pair_of<ST>(b0), c1 = pair_of<ST>(b1);
          b1 = fmaxf(fmaxf(b1, c1), fminf(b0, c0));
          b0 = fmaxf(b0, c0);
        }
      };
      merge(std::integral_constant<int, 0>{});
      merge(std::integral_constant<int, 1>{});
      merge(std::integral_constant<int, 2>{});
      merge(std::integral_constant<int, 3>{});
      merge(std::integral_constant<int, 4>{});
      const uint32_t gk = g < G ? order_key(a.group_top == 2 ? b0 + b1 : b0) : 0u;
      int rank = 0;
      for (int h = 0; h < G; ++h) {
        const uint32_t hk = (uint32_t)__builtin_amdgcn_readlane((int)gk, h << shift);
        rank += (hk > gk) | ((hk == gk) & (h < g));
      }
      const uint64_t stay = __ballot((g < G) & (rank < a.top_groups));
#pragma unroll
      for (int j = 0; j < PER; ++j) key[j] = ((stay >> gbit[j]) & 1) ? key[j] : 0u;
    }

    // Top-k: the wave's best value, then the lowest expert that has it.
    float my_r = 0.f, total = 0.f;
    int my_e = 0;
    for (int i = 0; i < k; ++i) {
      uint32_t best = key[0];
#pragma unroll
      for (int j = 1; j < PER; ++j) best = max(best, key[j]);
      best = wave_max_u32(best);
      int e = 0;
#pragma unroll
      for (int j = PER - 1; j >= 0; --j) {
        const uint64_t hit = __ballot(key[j] == best);
        e = hit ? j * 64 + __ffsll((unsigned long long)hit) - 1 : e;
      }
      e = __builtin_amdgcn_readfirstlane(e);
      float r = 0.f;
#pragma unroll
      for (int j = 0; j < PER; ++j) {
        const bool it = j * 64 + lane == e;
        r = it ? s[j] : r;
        key[j] = it ? 0u : key[j];
        if (TRAIN) pl[j] += it;
      }
      r = __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(r), e & 63));
      total += r;
      my_r = lane == i ? r : my_r;
      my_e = lane == i ? e : my_e;
    }
    if (lane < k) {
      a.topk_idx[(size_t)t * k + lane] = my_e;
      a.topk_w[(size_t)t * k + lane] = a.renorm ? a.scale * (my_r / (total + 1e-20f)) : a.scale * my_r;
    }
  }
};

// Tokens whose logits lie in `parts` parts at `in` [parts][T][E] (no bias yet), or, FINAL, as
// they are in a.logits; one wave per token.  TRAIN: this block's column of the sums over
// tokens, [E][blocks], waves added in order.
template <int PER, bool TRAIN, int WAVES>
__global__ __launch_bounds__(WAVES * 64) void score_finish_kernel(ScoreArgs a, int parts, bool final) {
  __shared__ float sel[WAVES][64 * PER];
  __shared__ double sum_p[TRAIN ? WAVES : 1][64 * PER];
  __shared__ int sum_l[TRAIN ? WAVES : 1][64 * PER];
  __shared__ double sum_z[WAVES];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int E = a.sh.E, T = a.sh.T;
  const size_t step = (size_t)T * E;
  Finisher<PER, TRAIN> f;
  f.init(a);
  float bias[PER];
#pragma unroll
  for (int j = 0; j < PER; ++j) bias[j] = (!final && a.b_router && f.live[j]) ? a.b_router[j * 64 + lane] : 0.f;
  const float* in = final ? a.logits : a.part;
  for (int t = blockIdx.x * WAVES + wave; t < T; t += gridDim.x * WAVES) {
    float l[PER];
    const float* row = in + (size_t)t * E;
#pragma unroll
    for (int j = 0; j < PER; ++j) l[j] = row[min(j * 64 + lane, E - 1)];
    for (int p = 1; p < parts; p += 4) {               // parts added in order, four loads at once
      float v[4][PER];
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int j = 0; j < PER; ++j) v[q][j] = row[min(p + q, parts - 1) * step + min(j * 64 + lane, E - 1)];
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int j = 0; j < PER; ++j) l[j] += p + q < parts ? v[q][j] : 0.f;
    }
#pragma unroll
    for (int j = 0; j < PER; ++j) l[j] = f.live[j] ? l[j] + bias[j] : -INFINITY;
    if (!final && a.logits) {
#pragma unroll
      for (int j = 0; j < PER; ++j)
        if (f.live[j]) a.logits[(size_t)t * E + j * 64 + lane] = l[j];
    }
    f.token(a, t, l, sel[wave]);
  }
  if constexpr (TRAIN) {
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      sum_p[wave][j * 64 + lane] = f.pq[j];
      sum_l[wave][j * 64 + lane] = f.pl[j];
    }
    if (lane == 0) sum_z[wave] = f.pz;
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += WAVES * 64) {
      double p = sum_p[0][e];
      int n = sum_l[0][e];
#pragma unroll
      for (int w = 1; w < WAVES; ++w) p += sum_p[w][e], n += sum_l[w][e];
      a.psum[(size_t)e * gridDim.x + blockIdx.x] = p;
      a.pload[(size_t)e * gridDim.x + blockIdx.x] = n;
    }
    if (threadIdx.x == 0) {
      double z = sum_z[0];
#pragma unroll
      for (int w = 1; w < WAVES; ++w) z += sum_z[w];
      a.pz[blockIdx.x] = z;
    }
  }
}

// ---------------------------------------------------------------------------
// Many tokens: 64 tokens x all experts (NE columns) per block, both operands through LDS in
// steps of 128 bytes of d; rows of 128 B with 16 B chunks at chunk ^ ((row >> 1) & 7) (16
// rows' reads of a chunk touch every bank once).  W_r goes by the MFMA's first operand, so a
// lane holds four neighbouring experts of a token.  bf16: MFMA 32x32x16; fp32: 32x32x2,
// lane half h taking chunk 2s + h of a row for slice s (both operands agree on the k of a
// slot).
// W_r comes from L2, two steps ahead; x from memory, five: 256 CUs need about
// 8 MB in flight to read at full rate, two steps of x were 4 MB.
// Eight waves, two per SIMD: waves 0-3 multiply the first half of each step, 4-7 the
// second, each over the whole tile, so LDS is read no more often than by four waves while
// one wave's reads run under the other's MFMAs; the halves add up at the end through LDS.
// 16384 tokens, d = 4096, 256 experts: 44 us, x read at 3.0 TB/s, 780 TFLOP/s.  Bound: each
// block also takes all of W_r from L2, 20480 cache lines at about one per ns in all; more
// tokens per block would halve that but leave CUs idle (256 blocks here).
// One part (d not split) and the logits wanted: they are written there, bias included; else
// to the workspace.  Finishing the tokens in this kernel measured slower: with so few
// waves a token took 5 us, the separate kernel has the waves to hide that.
// ---------------------------------------------------------------------------
constexpr int kRowsM = 64, kXStages = 6, kWStages = 3;

template <typename T, int NE>
__global__ __launch_bounds__(512, 1) void score_tile_kernel(ScoreArgs a, int parts) {
  constexpr int kKs = 128 / sizeof(T);                 // d per step
  constexpr int WN = NE == 256 ? 4 : 2, WM = 4 / WN;   // waves of a half over experts, tokens
  constexpr int MT = kRowsM / WM / 32, NT = NE / WN / 32;
  constexpr int kX = kRowsM * 128, kW = NE * 128, kWBase = kXStages * kX;
  constexpr int kWI = kW / 8192, L = 1 + kWI;          // 1 KB loads per wave and step
  constexpr int kPitch = NE + 4;                       // floats per token's logits in LDS
  constexpr int kLogits = kRowsM * kPitch * 4;
  constexpr int kStages = kWBase + kWStages * kW;
  constexpr int kLds = kStages > kLogits ? kStages : kLogits;
  static_assert(kX == 8192 && kW % 8192 == 0 && kLds <= 160 * 1024, "load plan");
  __shared__ __attribute__((aligned(1024))) uint8_t lds[kLds];

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), half = wave >> 2;
  const int wm = (wave & 3) / WN, wn = (wave & 3) % WN, fr = lane & 31, fc = lane >> 5;
  const int E = a.sh.E, tokens = a.sh.T, d = a.sh.d;
  const int part = blockIdx.y, t0 = blockIdx.x * kRowsM;
  const int steps = d / kKs;
  const int s0 = (int)((long)part * steps / parts), nk = (int)((long)(part + 1) * steps / parts) - s0;
  const uint32_t lds0 = (uint32_t)(uintptr_t)lds;
  const size_t pitch = (size_t)d * sizeof(T);
  if (part == 0 && blockIdx.x == 0 && threadIdx.x == 0) *a.done = 0u;

  // Loads: instruction i of wave w fills rows (8i + w) * 8 + lane / 8, chunk lane % 8.
  const int row0 = wave * 8 + (lane >> 3);
  const uint32_t chunk = ((lane & 7) ^ ((row0 >> 1) & 7)) << 4;
  const uint32_t x_off = (uint32_t)(min(row0, tokens - 1 - t0) * pitch) + chunk;
  uint32_t w_off[kWI];
#pragma unroll
  for (int i = 0; i < kWI; ++i) w_off[i] = (uint32_t)(min(i * 64 + row0, E - 1) * pitch) + chunk;
  const uint32_t swz = (fr >> 1) & 7;
  const uint8_t* x_base = static_cast<const uint8_t*>(a.x) + (size_t)t0 * pitch + (size_t)s0 * 128;
  const uint8_t* w_base = static_cast<const uint8_t*>(a.w) + (size_t)s0 * 128;
  // Steps past the last repeat it (into free stages).
  auto load_x = [&](int step, int stage) {
    dma16(x_base + (size_t)min(step, nk - 1) * 128, x_off, lds0 + stage * kX + wave * 1024);
  };
  auto load_w = [&](int i, int step, int stage) {
    dma16(w_base + (size_t)min(step, nk - 1) * 128, w_off[i], lds0 + kWBase + stage * kW + (i * 8 + wave) * 1024);
  };
  f32x16 acc[NT][MT];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int q = 0; q < 16; ++q) acc[n][m][q] = 0.f;

  u32x4 xa[2][MT], wb[2][NT];
  auto read = [&](int i, int stage_x, int stage_w) {   // slice i of this half of a step
    const uint32_t c = ((4 * half + 2 * i + fc) ^ swz) << 4;
#pragma unroll
    for (int m = 0; m < MT; ++m) xa[i][m] = ld16(lds + stage_x * kX + ((wm * MT * 32 + fr) * 128 + c) + m * 4096);
#pragma unroll
    for (int n = 0; n < NT; ++n)
      wb[i][n] = ld16(lds + kWBase + stage_w * kW + ((wn * NT * 32 + fr) * 128 + c) + n * 4096);
  };
  // Slice 0 of step t is in registers when it starts; slice 1 is read under slice 0's MFMAs
  // and the next step's slice 0 under slice 1's, with the loads between the MFMAs (all at
  // once they hold the waves up).  The barrier sits in the middle: the next step has landed,
  // everyone has read the last of this one.
#pragma unroll
  for (int s = 0; s < kXStages; ++s) load_x(s, s);
#pragma unroll
  for (int s = 0; s < kWStages; ++s)
#pragma unroll
    for (int i = 0; i < kWI; ++i) load_w(i, s, s);
  __builtin_amdgcn_s_waitcnt(wait_vm((kWStages - 1) * kWI));
  __syncthreads();
  read(0, 0, 0);
  int sx = 0, sw = 0;                                  // stages of step t
  constexpr int kM = NT * MT;
  auto mfma = [&](int i, int q) {
    const int n = q / MT, m = q % MT;
    if constexpr (sizeof(T) == 2) {
      acc[n][m] = mfma32_bf16(wb[i][n], xa[i][m], acc[n][m]);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        acc[n][m] = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(wb[i][n][j]), __uint_as_float(xa[i][m][j]),
                                                         acc[n][m], 0, 0, 0);
    }
  };
  for (int t = 0; t < nk; ++t) {
    const int sx1 = sx == kXStages - 1 ? 0 : sx + 1, sw1 = sw == kWStages - 1 ? 0 : sw + 1;
    read(1, sx, sw);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int q = 0; q < kM; ++q) mfma(0, q);
    __builtin_amdgcn_sched_barrier(0);
    // Step t + 1 landed: in flight may be only what step t - 1 issued (at first W's step 2).
    if (t == 0) __builtin_amdgcn_s_waitcnt(wait_vm_lgkm0(kWI));
    else __builtin_amdgcn_s_waitcnt(wait_vm_lgkm0(L));
    __syncthreads();
    read(0, sx1, sw1);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int q = 0; q < kM; ++q) {
      mfma(1, q);
#pragma unroll
      for (int j = q * L / kM; j < (q + 1) * L / kM; ++j) {
        if (j == 0) load_x(t + kXStages, sx);
        else load_w(j - 1, t + kWStages, sw);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    sx = sx1;
    sw = sw1;
  }
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");        // the repeated loads too
  __syncthreads();                                     // LDS free

  // Lane: token m * 32 + fr, experts n * 32 + 8 g + 4 fc .. + 3.  First half + second half.
  float* lg = reinterpret_cast<float*>(lds);
#pragma unroll
  for (int h = 1; h >= 0; --h) {
    if (half == h) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            const int e = (wn * NT + n) * 32 + 8 * g + 4 * fc, r = (wm * MT + m) * 32 + fr;
            f32x4* at = reinterpret_cast<f32x4*>(lg + r * kPitch + e);
            f32x4 v = {acc[n][m][4 * g], acc[n][m][4 * g + 1], acc[n][m][4 * g + 2], acc[n][m][4 * g + 3]};
            if (h == 0) v += *at;
            *at = v;
          }
    }
    __syncthreads();
  }
  const bool final = parts == 1 && a.logits;
  float* out = final ? a.logits : a.part + (size_t)part * tokens * E;
  float bias[NE / 64];
#pragma unroll
  for (int j = 0; j < NE / 64; ++j)
    bias[j] = (final && a.b_router && j * 64 + lane < E) ? a.b_router[j * 64 + lane] : 0.f;
#pragma unroll
  for (int i = 0; i < kRowsM / 8; ++i) {
    const int r = i * 8 + wave, t = t0 + r;
#pragma unroll
    for (int j = 0; j < NE / 64; ++j)
      if (t < tokens && j * 64 + lane < E) out[(size_t)t * E + j * 64 + lane] = lg[r * kPitch + j * 64 + lane] + bias[j];
  }
}

// The sums over blocks (at most 256) in a fixed order: a wave per expert, its column read at
// once.  The block that finishes last (a counter that the logits kernel cleared; agent-wide
// release and acquire around it) has all of them and writes the losses.  8 us whatever the
// sizes: three dependent trips to memory.
__global__ __launch_bounds__(1024) void score_reduce_kernel(ScoreArgs a, int blocks) {
  __shared__ bool last;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, E = a.sh.E;
  const int e = blockIdx.x * 16 + wave;
  auto total = [&](double v) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
    return v;
  };
  if (e < E) {
    double p = 0.0;
    int n = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int b = i * 64 + lane;
      if (b < blocks) {
        p += a.psum[(size_t)e * blocks + b];
        n += a.pload[(size_t)e * blocks + b];
      }
    }
    p = total(p) / a.sh.T;
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) n += __shfl_xor(n, o);
    if (lane == 0) {
      if (a.prob_mean) a.prob_mean[e] = (float)p;
      if (a.load) a.load[e] = n;
      a.share[e] = p * n;
    }
  }
  if (!a.aux && !a.z_loss) return;
  // The release below waits for its own wave's stores only, and a barrier for none: each wave
  // has its share in L2 before it arrives there.
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();
  if (threadIdx.x == 0)
    last = __hip_atomic_fetch_add(a.done, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) == gridDim.x - 1;
  __syncthreads();
  if (!last || wave != 0) return;
  double x = 0.0, z = 0.0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int j = i * 64 + lane;
    if (j < E) x += __hip_atomic_load(a.share + j, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    if (j < blocks) z += a.pz[j];
  }
  x = total(x);
  z = total(z);
  if (lane == 0) {
    if (a.aux) *a.aux = (float)(x * E / ((double)a.sh.T * a.sh.k));
    if (a.z_loss) *a.z_loss = (float)(z / a.sh.T);
  }
}

template <typename T>
static void launch_typed(const ScoreArgs& a, bool train, hipStream_t s) {
  const ScoreShape& h = a.sh;
  const int parts = score_parts(h);
  const bool tiled = score_tiled(h);
  if (tiled) {
    const dim3 grid((h.T + kRowsM - 1) / kRowsM, parts);
    if (h.E <= 64) score_tile_kernel<T, 64><<<grid, 512, 0, s>>>(a, parts);
    else if (h.E <= 128) score_tile_kernel<T, 128><<<grid, 512, 0, s>>>(a, parts);
    else if (h.E <= 192) score_tile_kernel<T, 192><<<grid, 512, 0, s>>>(a, parts);
    else score_tile_kernel<T, 256><<<grid, 512, 0, s>>>(a, parts);
  } else {
    const dim3 grid((h.T + 15) / 16, (h.E + 63) / 64, parts);
    score_logits_kernel<T><<<grid, 256, 0, s>>>(static_cast<const T*>(a.x), static_cast<const T*>(a.w), h.T,
                                               h.d, h.E, parts, a.part, a.done);
  }
  // Blocks of 4 waves while they spread over the chip, of 16 where tokens abound (whole calls,
  // d = 4096, 256 experts: 512 tokens 30 and 32 us, 1024 tokens 31 and 30, 4096 tokens 42 and 37).
  const bool big = h.T >= 1024, final = tiled && parts == 1 && a.logits;
  const int nb = std::min(256, (h.T + (big ? 15 : 3)) / (big ? 16 : 4));
  auto finish = [&](auto per) {
    constexpr int PER = decltype(per)::value;
    if (train && big) score_finish_kernel<PER, true, 16><<<nb, 1024, 0, s>>>(a, parts, final);
    else if (train) score_finish_kernel<PER, true, 4><<<nb, 256, 0, s>>>(a, parts, final);
    else if (big) score_finish_kernel<PER, false, 16><<<nb, 1024, 0, s>>>(a, parts, final);
    else score_finish_kernel<PER, false, 4><<<nb, 256, 0, s>>>(a, parts, final);
  };
  if (h.E <= 64) finish(std::integral_constant<int, 1>{});
  else if (h.E <= 128) finish(std::integral_constant<int, 2>{});
  else finish(std::integral_constant<int, 4>{});
  if (train) score_reduce_kernel<<<(h.E + 15) / 16, 1024, 0, s>>>(a, nb);
}

hipError_t launch_score(const ScoreArgs& a, hipStream_t s) {
  const bool train = a.load || a.prob_mean || a.aux || a.z_loss;
  if (a.sh.bf16) launch_typed<uint16_t>(a, train, s);
  else launch_typed<float>(a, train, s);
  return hipGetLastError();
}

}  // namespace moe
