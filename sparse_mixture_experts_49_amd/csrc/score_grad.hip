// Gradients of the scored router on gfx950.
//
// For each token, with g = d topk_w, chosen scores r_j = s[idx_j], S = sum r + 1e-20:
//   dr_j = scale g_j, or renormalised scale sum_i r_i (g_j - g_i) / S^2
//   dq_e = d_aux E load_e / (T k) / T          (q = s / sum s; load is a constant)
//   softmax: ds = dr + dq;                       dl = s (ds - sum ds s)
//   sigmoid: ds = dr + (dq - sum dq q) / sum s;  dl = ds s (1 - s) = (dr s + (dq - sum dq q) q) (1 - s)
//   dl += d_z (2 / T) lse softmax(l)
// The differences with a sum over all experts are formed as of_leader says.
// and d_b = sum_t dl, d_x = dl W_r, d_W = dl^T x.
//
// bf16 layers: x and W_r go to the bf16 MFMA as they are and dl as a sum of bf16 terms,
// dl = hi + mid (+ lo): two keep 17 bits, enough under d_x's rounding to bf16, three keep
// all of fp32's for the fp32 d_W.  dl itself is kept in fp32 and split where it is multiplied
// (written out as terms it is half as many bytes again and more cache lines).
#include <algorithm>
#include <type_traits>

#include "device_common.h"
#include "score.h"

namespace moe {

__host__ __device__ static int up_to(int v, int m) { return (v + m - 1) / m * m; }

// Column blocks of the products: 256 columns of d each.
constexpr int kGradCols = 256, kGradRows = 128, kGradK = 32;

int score_grad_slices(const ScoreShape& s) {
  if (s.bf16) {
    // Blocks of kGradRows experts x 256 columns; slices of at least 128 tokens until every
    // CU has a block (its LDS holds no second one).
    const long tiles = (long)((s.E + kGradRows - 1) / kGradRows) * ((s.d + kGradCols - 1) / kGradCols);
    return (int)std::max(1L, std::min({32L, (long)(s.T + 127) / 128, 256 / tiles}));
  }
  // fp32: tiles of 16 experts x 64 columns per wave; slices of at least 64 tokens until
  // 2048 waves run.
  const long tiles = (long)((s.E + 15) / 16) * (s.d / 64);
  return (int)std::max(1L, std::min({16L, (long)(s.T + 63) / 64, 2048 / tiles}));
}

// Tokens per tile of the logit-gradient kernel (blocks of 4 or 16 waves): 64 and 256 experts,
// tiles of 16 and 64, us: 4096 tokens 8.2 and 9.4, 11.2 and 14.4; 8192 tokens 10.7 and 9.8, 15.4
// and 15.3; 16384 tokens 16 and 11, 26 and 18.
static int grad_tile(int T) { return T >= 8192 ? 64 : 16; }
static int grad_blocks(int T) {
  const int tile = grad_tile(T);
  return std::min(256, (T + tile - 1) / tile);
}

// Workspace of the logit gradients: fp32 [T up to 32][E up to whole tiles of the d_W product],
// zeros behind T and E.
static int dl_pitch(int E) { return E <= 64 ? 64 : up_to(E, kGradRows); }

size_t score_dl_bytes(const ScoreShape& s) { return (size_t)up_to(s.T, kGradK) * dl_pitch(s.E) * 4; }
int score_grad_sum_blocks(int T) { return grad_blocks(T); }

// The v of the expert with more than `half` (half of all) of a token's score, 0 if none has.
// v_i - sum_j v_j s_j does not change when a constant is taken off every v.  With the leader's
// own value taken off, its difference is the small sum of what the others get instead of two
// nearly equal numbers, and no other's is less exact; without a leader nothing cancels.
template <int PER>
__device__ __forceinline__ float of_leader(const float (&s)[PER], float half, const float (&v)[PER]) {
  float u = 0.f;
  bool mine = false;
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const bool it = s[j] > half;                         // one expert at most
    u = it ? v[j] : u;
    mine |= it;
  }
  const uint64_t at = __ballot(mine);
  uint32_t c = (uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(u), (__ffsll((unsigned long long)at) - 1) & 63);
  c = at ? c : 0u;
  return __uint_as_float((c & 0x7f800000u) == 0x7f800000u ? 0u : c);   // infinite: off nothing
}

// dl of tiles of TT tokens, one at a time per wave, lane l the experts l, l + 64, ... and for
// the chosen ones lane q < k the q-th.  Bound by instruction issue, so straight-line: experts
// behind E and slots behind k carry zeros, what depends on an argument is computed with 0 where
// it is absent.  16384 tokens, 256 experts, k = 8: 24 us for 34 MB.
template <int PER, int TT, bool SIGMOID>
__global__ __launch_bounds__(TT * 16) void score_dlogits_kernel(ScoreGradArgs a) {
  constexpr int WAVES = TT / 4, kThreads = TT * 16, kPitch = 64 * PER;
  __shared__ double sum_b[WAVES][64 * PER];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int E = a.sh.E, T = a.sh.T, k = a.sh.k;
  const float aux = a.d_aux ? *a.d_aux : 0.f, z = a.d_z ? *a.d_z * 2.f / T : 0.f;
  float dq[PER];
  bool live[PER];
  double pb[PER];
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const int e = j * 64 + lane;
    live[j] = e < E;
    dq[j] = (a.d_aux && live[j]) ? (float)((double)aux * E * a.load[e] / ((double)T * k) / T) : 0.f;
    pb[j] = 0.0;
  }
  for (int t0 = blockIdx.x * TT; t0 < T; t0 += gridDim.x * TT) {
    for (int t = t0 + wave; t < min(t0 + TT, T); t += WAVES) {
      float l[PER], p[PER], s[PER], rest[SIGMOID ? PER : 1];   // rest: 1 - s
#pragma unroll
      for (int j = 0; j < PER; ++j) l[j] = a.logits[(size_t)t * E + min(j * 64 + lane, E - 1)];
      int idx = a.topk_idx[(size_t)t * k + min(lane, k - 1)];
      float g = a.d_topk_w ? a.d_topk_w[(size_t)t * k + min(lane, k - 1)] : 0.f;
      idx = (lane < k && (uint32_t)idx < (uint32_t)E) ? idx : -1;
      g = idx >= 0 ? g : 0.f;
#pragma unroll
      for (int j = 0; j < PER; ++j) l[j] = live[j] ? l[j] : -INFINITY;
      float zl = 0.f;                                  // d_z (2 / T) lse
      if (!SIGMOID || a.d_z) {
        float m = l[0], tot = 0.f;
#pragma unroll
        for (int j = 1; j < PER; ++j) m = fmaxf(m, l[j]);
        m = wave_max_f(m);
        m = m == -INFINITY ? 0.f : m;
#pragma unroll
        for (int j = 0; j < PER; ++j) tot += p[j] = exp_f32(l[j] - m);
        tot = wave_sum_f(tot);
        const float r_tot = tot > 0.f ? 1.f / tot : tot != tot ? tot : 0.f;
#pragma unroll
        for (int j = 0; j < PER; ++j) p[j] *= r_tot;
        if (a.d_z) zl = z * fmaf(__builtin_amdgcn_logf(tot), 0.69314718055994530942f, m);
      } else {
#pragma unroll
        for (int j = 0; j < PER; ++j) p[j] = 0.f;
      }
#pragma unroll
      for (int j = 0; j < PER; ++j) {
        if constexpr (SIGMOID) sigmoid_pair(l[j], s[j], rest[j]);
        else s[j] = p[j];
      }
      // Chosen scores and the gradients of the raw weights, lane q those of choice q.
      float r = 0.f;
#pragma unroll
      for (int j = 0; j < PER; ++j) {
        const float v = __uint_as_float(
            (uint32_t)__builtin_amdgcn_ds_bpermute((idx & 63) << 2, (int)__float_as_uint(s[j])));
        r = idx >> 6 == j ? v : r;                     // idx -1: none
      }
      if (a.renorm) {
        // g_j S - sum_i g_i r_i by differences: with one choice, or equal gradients, 0.
        const float rS = 1.f / (wave_sum_f(r) + 1e-20f);
        float v = 1e-20f * g;
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const float rq = __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(r), q));
          const float gq = __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(g), q));
          v = fmaf(rq, g - gq, v);
        }
        g = a.scale * (v * rS) * rS;
      } else {
        g *= a.scale;
      }
      float ds[PER];
#pragma unroll
      for (int j = 0; j < PER; ++j) ds[j] = 0.f;
#pragma unroll
      for (int q = 0; q < 8; ++q) {                    // k is at most 8
        const int iq = __builtin_amdgcn_readlane(idx, q);
        const float gq = __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(g), q));
#pragma unroll
        for (int j = 0; j < PER; ++j) ds[j] += iq == j * 64 + lane ? gq : 0.f;
      }
      float dl[PER];
      if constexpr (SIGMOID) {
        if (a.d_aux) {
          float cq = 0.f, ss = 0.f;
#pragma unroll
          for (int j = 0; j < PER; ++j) ss += s[j];
          ss = wave_sum_f(ss);
          const float rs = 1.f / (ss < kLeastSum ? kLeastSum : ss), c = of_leader(s, 0.5f * ss, dq);
          float q[PER];                                // s / sum s, where ds itself may overflow
#pragma unroll
          for (int j = 0; j < PER; ++j) {
            q[j] = s[j] * rs;
            cq = fmaf(dq[j] - c, q[j], cq);
          }
          cq = wave_sum_f(cq);
#pragma unroll
          for (int j = 0; j < PER; ++j) dl[j] = (dq[j] - c - cq) * q[j];
        } else {
#pragma unroll
          for (int j = 0; j < PER; ++j) dl[j] = 0.f;
        }
#pragma unroll
        for (int j = 0; j < PER; ++j) dl[j] = fmaf(ds[j], s[j], dl[j]) * rest[j];
      } else {
        float cs = 0.f;
#pragma unroll
        for (int j = 0; j < PER; ++j) ds[j] += dq[j];
        const float c = of_leader(s, 0.5f, ds);
#pragma unroll
        for (int j = 0; j < PER; ++j) {
          ds[j] -= c;
          cs = fmaf(ds[j], s[j], cs);
        }
        cs = wave_sum_f(cs);
#pragma unroll
        for (int j = 0; j < PER; ++j) dl[j] = s[j] * (ds[j] - cs);
      }
#pragma unroll
      for (int j = 0; j < PER; ++j) {
        dl[j] = live[j] ? fmaf(zl, p[j], dl[j]) : 0.f;
        pb[j] += (double)dl[j];
        a.dl[(size_t)t * kPitch + j * 64 + lane] = dl[j];
      }
      if (a.d_logits) {
#pragma unroll
        for (int j = 0; j < PER; ++j)
          if (live[j]) a.d_logits[(size_t)t * E + j * 64 + lane] = dl[j];
      }
    }
    // The last tile also clears the rows behind T (the end of d_W's last step).
    if (t0 + TT >= T)
      for (int i = threadIdx.x; i < (up_to(T, kGradK) - T) * kPitch; i += kThreads) a.dl[(size_t)T * kPitch + i] = 0.f;
  }
  if (a.d_b) {
#pragma unroll
    for (int j = 0; j < PER; ++j) sum_b[wave][j * 64 + lane] = pb[j];
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += kThreads) {
      double p = sum_b[0][e];
#pragma unroll
      for (int w = 1; w < WAVES; ++w) p += sum_b[w][e];
      a.pb[(size_t)e * gridDim.x + blockIdx.x] = p;
    }
  }
}

// d_b: a wave per expert, its column of block sums (at most 256) read at once.
__global__ __launch_bounds__(256) void score_db_kernel(const double* __restrict__ pb, int blocks,
                                                       int E, float* __restrict__ d_b) {
  const int lane = threadIdx.x & 63, e = blockIdx.x * 4 + (threadIdx.x >> 6);
  if (e >= E) return;
  double p = 0.0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int b = i * 64 + lane;
    if (b < blocks) p += pb[(size_t)e * blocks + b];
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) p += __shfl_xor(p, o);
  if (lane == 0) d_b[e] = (float)p;
}

// Two neighbouring fp32 values to one word of each of TERMS bf16 fragments.
template <int TERMS>
__device__ __forceinline__ void split_pair(float u, float v, uint32_t (&out)[TERMS]) {
#pragma unroll
  for (int q = 0; q < TERMS; ++q) {
    out[q] = pack_bf16x2(u, v);
    u -= __uint_as_float(out[q] << 16);
    v -= __uint_as_float(out[q] & 0xffff0000u);
  }
}

// The MFMA wants 8 values along k per lane from both operands.  The products' B (W_r by
// expert, x by token) has its rows along n, so a lane reads the pair of neighbouring columns
// 2l, 2l + 1 from 8 rows (a row's 32 pairs are 128 contiguous bytes) and splits the words into
// two fragments, even and odd columns.  As the first operand they make a lane's accumulators,
// even and odd together, 8 neighbouring columns of one row: column 16 g + 8 fc of 64.
__device__ __forceinline__ uint32_t even_pair(uint32_t w0, uint32_t w1) {
  return __builtin_amdgcn_perm(w1, w0, 0x05040100);
}
__device__ __forceinline__ uint32_t odd_pair(uint32_t w0, uint32_t w1) {
  return __builtin_amdgcn_perm(w1, w0, 0x07060302);
}
__device__ __forceinline__ void columns8(const f32x16& u, const f32x16& v, int g, f32x4& lo, f32x4& hi) {
  lo = f32x4{u[4 * g], v[4 * g], u[4 * g + 1], v[4 * g + 1]};
  hi = f32x4{u[4 * g + 2], v[4 * g + 2], u[4 * g + 3], v[4 * g + 3]};
}

// ---------------------------------------------------------------------------
// d_x[t] = dl[t] W_r.  k is the experts, at most 256, so W_r stays in registers: a wave has 64
// columns of it for every expert (NE / 2 registers), a block of eight 512, and tiles of 32
// tokens stream past.  The block splits a tile of dl into its two bf16 terms once, into LDS
// (rows of 2 NE bytes per term, 16 B chunks at chunk ^ f(row) such that 16 rows' reads of one
// touch every bank once), two tiles in turn with one barrier each; the next tile's dl is on its
// way meanwhile.  16384 x 4096, 256 experts: 77 us, 0.89 PFLOP/s of the two terms; the MFMAs
// take 59% of the waves' time, the rest is reading W_r (once per block, 8 us) and the stores.
// ---------------------------------------------------------------------------
constexpr int kDxCols = 512, kDxRows = 32;

template <int NE>
__global__ __launch_bounds__(512, 2) void score_dx_bf16_kernel(const float* __restrict__ dl, int pitch,
                                                               const uint16_t* __restrict__ w, int T, int d,
                                                               int E, int groups, uint16_t* __restrict__ d_x) {
  constexpr int kTerm = kDxRows * NE * 2, kChunks = NE / 8, kUnits = kDxRows * kChunks;
  constexpr int kPer = (kUnits + 511) / 512;           // chunks of 8 values per thread
  constexpr int kSlices = NE / 16;
  // Rows of whole 256 B start at the same bank, of odd multiples of 128 B at two in turn.
  auto swz = [](int r) { return NE % 128 == 0 ? r & 15 : (r >> 1) & 7; };
  __shared__ __attribute__((aligned(1024))) uint8_t lds[2 * 2 * kTerm];
  const int lane = threadIdx.x & 63, fr = lane & 31, fc = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int group = blockIdx.x % groups, c0 = (blockIdx.x / groups) * kDxCols + wave * 64;
  const int tiles = (T + kDxRows - 1) / kDxRows;
  const bool active = c0 < d;                          // d is a multiple of 128

  u32x4 b[kSlices][2];
  {
    const uint16_t* col = w + (active ? c0 : 0) + 2 * fr;
#pragma unroll
    for (int s = 0; s < kSlices; ++s) {
      uint32_t v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int e = s * 16 + fc * 8 + j;
        v[j] = *reinterpret_cast<const uint32_t*>(col + (size_t)min(e, E - 1) * d);
        v[j] = e < E ? v[j] : 0u;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) b[s][0][j] = even_pair(v[2 * j], v[2 * j + 1]), b[s][1][j] = odd_pair(v[2 * j], v[2 * j + 1]);
    }
  }

  f32x4 next[kPer][2];
  auto fetch = [&](int tile) {                         // dl has whole tiles of rows, NE columns or more
    const float* row = dl + (size_t)min(tile, tiles - 1) * kDxRows * pitch;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int u = i * 512 + (int)threadIdx.x, r = u / kChunks, c = u % kChunks;
      next[i][0] = next[i][1] = f32x4{0.f, 0.f, 0.f, 0.f};
      if (u < kUnits) {
        next[i][0] = *reinterpret_cast<const f32x4*>(row + (size_t)r * pitch + c * 8);
        next[i][1] = *reinterpret_cast<const f32x4*>(row + (size_t)r * pitch + c * 8 + 4);
      }
    }
  };
  auto put = [&](int buffer) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int u = i * 512 + (int)threadIdx.x, r = u / kChunks, c = u % kChunks;
      if (u >= kUnits) continue;
      u32x4 q[2];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const f32x4 f = next[i][j >> 1];
        uint32_t o[2];
        split_pair<2>(f[2 * (j & 1)], f[2 * (j & 1) + 1], o);
        q[0][j] = o[0], q[1][j] = o[1];
      }
      uint8_t* at = lds + buffer * 2 * kTerm + r * NE * 2 + ((c ^ swz(r)) << 4);
      *reinterpret_cast<u32x4*>(at) = q[0];
      *reinterpret_cast<u32x4*>(at + kTerm) = q[1];
    }
  };
  fetch(group);
  put(0);
  fetch(group + groups);
  __syncthreads();
  int buffer = 0;
  for (int tile = group; tile < tiles; tile += groups, buffer ^= 1) {
    // The two waves of a SIMD do this before and after their MFMAs: one's runs under the
    // other's.
    if (wave < 4) {
      put(buffer ^ 1);
      fetch(tile + 2 * groups);
    }
    f32x16 acc[2];
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int q = 0; q < 16; ++q) acc[n][q] = 0.f;
    const uint8_t* base = lds + buffer * 2 * kTerm + fr * NE * 2;
    u32x4 f[2][2];                                     // [slice % 2][hi, mid]
    auto read = [&](int s) {
      const uint32_t at = ((2 * s + fc) ^ swz(fr)) << 4;
      f[s % 2][0] = ld16(base + at);
      f[s % 2][1] = ld16(base + kTerm + at);
    };
    read(0);
#pragma unroll
    for (int s = 0; s < kSlices; ++s) {
      if (s + 1 < kSlices) read(s + 1);
#pragma unroll
      for (int q = 1; q >= 0; --q)
#pragma unroll
        for (int n = 0; n < 2; ++n) acc[n] = mfma32_bf16(b[s][n], f[s % 2][q], acc[n]);
      __builtin_amdgcn_sched_barrier(0);
    }
    if (wave >= 4) {
      put(buffer ^ 1);
      fetch(tile + 2 * groups);
    }
    const int t = tile * kDxRows + fr;
    if (active && t < T) {
      uint16_t* o = d_x + (size_t)t * d + c0 + 8 * fc;
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        f32x4 lo, hi;
        columns8(acc[0], acc[1], g, lo, hi);
        st16(o + 16 * g, u32x4{pack_bf16x2(lo[0], lo[1]), pack_bf16x2(lo[2], lo[3]),
                               pack_bf16x2(hi[0], hi[1]), pack_bf16x2(hi[2], hi[3])});
      }
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------
// d_W[e][c] = sum_t dl[t][e] x[t][c]: A = dl, fp32 and multiplied as three bf16 terms, B = x,
// one slice of the tokens per block.  Block 64 MT experts x 256 columns, k in
// steps of 32 through four LDS stages, four waves as 2 x 2, one per SIMD.  All work but the
// MFMAs runs in their shadow: while a slice of 16 k is multiplied, the next one's fragments
// are made from words in registers, the words of the one after are read from LDS, and the
// loads of four steps ahead are issued.  One barrier per step.  16384 x 4096, 256 experts: 111 to
// 118 us by the box, 0.9 PFLOP/s of the three terms.  Nothing waits long: without the splitting
// 98 us, without the LDS reads 105; the chip's clock falls to 1.9 GHz under it, at which the
// MFMAs alone are busy 45% of the time.
//
// Both operands have their rows (tokens) along k, so a lane reads single words of 8 rows: of dl
// its expert's, of x its pair of columns.  LDS: rows of 256 MT and 512 B, their 128 B parts at
// part ^ ((row >> 3) & 1) so that the two lane halves (rows 8 apart) read different banks.
// ---------------------------------------------------------------------------
template <int MT>
__global__ __launch_bounds__(256, 1) void score_dw_bf16_kernel(
    const float* __restrict__ A, int a_pitch, const uint16_t* __restrict__ B, int T, int d, int E,
    int slices, float* __restrict__ out) {
  constexpr int S = 4, TERMS = 3, kRows = 64 * MT;
  constexpr int kA = kRows * 128, kStage = kA + kGradK * 512;
  constexpr int kAI = kA / 4096, kBI = 4, L = kAI + kBI;   // 1 KB loads per wave and step
  constexpr int kM = TERMS * 4 * MT;                   // MFMAs per slice
  static_assert(S * kStage <= 160 * 1024, "load plan");
  __shared__ __attribute__((aligned(1024))) uint8_t lds[S * kStage];
  const int lane = threadIdx.x & 63, fr = lane & 31, fc = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave >> 1, wn = wave & 1;
  // Slices fastest: with 8 of them the blocks of an XCD share one's dl and x in its L2.
  const int sl = blockIdx.x, n0 = blockIdx.y * kGradCols, m0 = blockIdx.z * kRows;
  const int steps = (T + kGradK - 1) / kGradK;
  const int s0 = (int)((long)sl * steps / slices), nk = (int)((long)(sl + 1) * steps / slices) - s0;
  const uint32_t lds0 = (uint32_t)(uintptr_t)lds;

  // A: load i of wave w fills 1 KB of rows of 256 MT bytes.
  constexpr int kALanes = 16 * MT;                     // lanes per row
  const float* a_base = A + (size_t)s0 * kGradK * a_pitch + m0;
  uint32_t a_off[kAI];
#pragma unroll
  for (int i = 0; i < kAI; ++i) {
    const int row = (i * 4 + wave) * (64 / kALanes) + lane / kALanes;
    a_off[i] = (uint32_t)row * (uint32_t)a_pitch * 4u + (((lane % kALanes) ^ (((row >> 3) & 1) << 3)) << 4);
  }
  // B: load i of wave w fills rows 2 (4 i + w) + lane / 32; rows past the last repeat it (A is
  // 0 there), columns past d wrap to the tile's first half (not stored).
  const uint8_t* b_tile = reinterpret_cast<const uint8_t*>(B + (size_t)s0 * kGradK * d + n0);
  auto load = [&](int i, int step, int stage) {
    const uint32_t base = lds0 + stage * kStage;
    const int s = min(step, nk - 1);
    if (i < kAI) {
      dma16(a_base + (size_t)s * kGradK * a_pitch, a_off[i < kAI ? i : 0], base + (i * 4 + wave) * 1024);
    } else {
      const int j = i - kAI, r = 2 * (j * 4 + wave) + (lane >> 5);
      int c = (lane & 31) ^ (((r >> 3) & 1) << 3);
      if (n0 + c * 8 >= d) c -= 16;
      const int row = min(r, T - 1 - (s0 + s) * kGradK);
      dma16(b_tile + (size_t)s * kGradK * d * 2, (uint32_t)(row * d + c * 8) * 2u,
            base + kA + (j * 4 + wave) * 1024);
    }
  };

  f32x16 acc[4][MT];                                   // [column group: 2 * (64 columns) + odd][m]
#pragma unroll
  for (int n = 0; n < 4; ++n)
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int q = 0; q < 16; ++q) acc[n][m][q] = 0.f;
  const uint32_t a_lane = 8 * fc * kRows * 4 + fr * 4, b_lane = kA + 8 * fc * 512 + fr * 4;
  float raw[MT][8];                                    // dl, 8 rows of an expert
  uint32_t pairs[2][8];                                // x, 8 rows of a pair of columns
  u32x4 xa[2][MT][TERMS], b[2][4];
  // Slice h of a stage: k 16 h + 8 fc .. + 7.
  auto read_a = [&](int stage, int h, int i) {
    const int m = i / 8, j = i % 8;
    raw[m][j] = *reinterpret_cast<const float*>(lds + stage * kStage + a_lane + (16 * h + j) * kRows * 4 +
                                                ((wm * MT + m) ^ fc) * 128);
  };
  auto read_b = [&](int stage, int h, int i) {         // i: 8 rows of two column groups
    const int n = i / 8, j = i % 8;
    pairs[n][j] = *reinterpret_cast<const uint32_t*>(lds + stage * kStage + b_lane + (16 * h + j) * 512 +
                                                     ((wn * 2 + n) ^ fc) * 128);
  };
  auto make_a = [&](u32x4 (&to)[MT][TERMS], int i) {
    const int m = i / 4, j = i % 4;
    uint32_t o[TERMS];
    split_pair<TERMS>(raw[m][2 * j], raw[m][2 * j + 1], o);
#pragma unroll
    for (int q = 0; q < TERMS; ++q) to[m][q][j] = o[q];
  };
  auto make_b = [&](u32x4 (&to)[4], int i) {
    const int n = i / 4, j = i % 4;
    to[2 * n][j] = even_pair(pairs[n][2 * j], pairs[n][2 * j + 1]);
    to[2 * n + 1][j] = odd_pair(pairs[n][2 * j], pairs[n][2 * j + 1]);
  };

#pragma unroll
  for (int s = 0; s < S; ++s)
#pragma unroll
    for (int i = 0; i < L; ++i) load(i, s, s);
  __builtin_amdgcn_s_waitcnt(wait_vm((S - 1) * L));
  __syncthreads();
#pragma unroll
  for (int h = 0; h < 2; ++h) {                        // slice 0 as fragments, slice 1 as words
#pragma unroll
    for (int i = 0; i < 8 * MT; ++i) read_a(0, h, i);
#pragma unroll
    for (int i = 0; i < 16; ++i) read_b(0, h, i);
    if (h == 0) {
#pragma unroll
      for (int i = 0; i < 4 * MT; ++i) make_a(xa[0], i);
#pragma unroll
      for (int i = 0; i < 8; ++i) make_b(b[0], i);
    }
  }
  int st = 0;
  for (int t = 0; t < nk; ++t) {
    const int st1 = st == S - 1 ? 0 : st + 1;
    __builtin_amdgcn_s_waitcnt(wait_vm_lgkm0((S - 2) * L));    // step t + 1 landed, step t read
    __syncthreads();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      // First third: the next slice's dl; second: its x, and the dl words of the one after;
      // last: their x words.
#pragma unroll
      for (int i = 0; i < kM; ++i) {                   // small terms first
        constexpr int kThird = kM / 3;
        const int q = TERMS - 1 - i / (4 * MT), n = i / MT % 4, m = i % MT, j = i % kThird;
        acc[n][m] = mfma32_bf16(b[h][n], xa[h][m][q], acc[n][m]);
        if (i < kThird) {
#pragma unroll
          for (int u = j * 4 * MT / kThird; u < (j + 1) * 4 * MT / kThird; ++u) make_a(xa[h ^ 1], u);
        } else if (i < 2 * kThird) {
#pragma unroll
          for (int u = j * 8 / kThird; u < (j + 1) * 8 / kThird; ++u) make_b(b[h ^ 1], u);
#pragma unroll
          for (int u = j * 8 * MT / kThird; u < (j + 1) * 8 * MT / kThird; ++u) read_a(st1, h, u);
        } else {
#pragma unroll
          for (int u = j * 16 / kThird; u < (j + 1) * 16 / kThird; ++u) read_b(st1, h, u);
        }
        const int at = h * kM + i;
#pragma unroll
        for (int u = at * L / (2 * kM); u < (at + 1) * L / (2 * kM); ++u) load(u, t + S, st);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    st = st1;
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");     // no load outlives its LDS
#pragma unroll
  for (int n = 0; n < 2; ++n)
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const int r = m0 + (wm * MT + m) * 32 + fr;
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const int col = n0 + wn * 128 + n * 64 + 16 * g + 8 * fc;
        f32x4 lo, hi;
        columns8(acc[2 * n][m], acc[2 * n + 1][m], g, lo, hi);
        if (r >= E || col >= d) continue;
        float* o = out + ((size_t)sl * E + r) * d + col;
        *reinterpret_cast<f32x4*>(o) = lo;
        *reinterpret_cast<f32x4*>(o + 4) = hi;
      }
    }
}

// fp32 layers: d_x tile of 16 tokens x 64 columns per wave: k-slot q of MFMA i is expert e0 + 4 i + q.
__global__ __launch_bounds__(256) void score_dx_kernel(const float* __restrict__ dl, int pitch,
                                                       const float* __restrict__ w, int tokens, int d,
                                                       int E, float* __restrict__ d_x) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, fr = lane & 15, fc = lane >> 4;
  const int t0 = blockIdx.x * 16, c0 = (blockIdx.y * 4 + wave) * 64;
  if (c0 >= d) return;
  const int t = min(t0 + fr, tokens - 1);
  f32x4 acc[4] = {};
  for (int e0 = 0; e0 < E; e0 += 4) {
    const int e = e0 + fc;
    const float a = e < E ? dl[(size_t)t * pitch + e] : 0.f;
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      const float b = e < E ? w[(size_t)e * d + c0 + n * 16 + fr] : 0.f;
      acc[n] = mfma_f32(a, b, acc[n]);
    }
  }
#pragma unroll
  for (int n = 0; n < 4; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = t0 + 4 * fc + i;
      if (row >= tokens) continue;
      d_x[(size_t)row * d + c0 + n * 16 + fr] = acc[n][i];
    }
}

// d_w_router tile of 16 experts x 64 columns per wave over one slice of the tokens.
__global__ __launch_bounds__(256) void score_dw_kernel(const float* __restrict__ dl, int pitch,
                                                       const float* __restrict__ x, int tokens, int d,
                                                       int E, int slices, float* __restrict__ out) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, fr = lane & 15, fc = lane >> 4;
  const int e0 = blockIdx.x * 16, c0 = (blockIdx.y * 4 + wave) * 64, sl = blockIdx.z;
  if (c0 >= d) return;
  const int ta = (int)((long)sl * tokens / slices), tb = (int)((long)(sl + 1) * tokens / slices);
  const int e = min(e0 + fr, E - 1);
  f32x4 acc[4] = {};
  for (int t0 = ta; t0 < tb; t0 += 4) {
    const int t = t0 + fc;
    const float a = t < tb ? dl[(size_t)t * pitch + e] : 0.f;
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      const float b = t < tb ? x[(size_t)t * d + c0 + n * 16 + fr] : 0.f;
      acc[n] = mfma_f32(a, b, acc[n]);
    }
  }
#pragma unroll
  for (int n = 0; n < 4; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = e0 + 4 * fc + i;
      if (row < E) out[((size_t)sl * E + row) * d + c0 + n * 16 + fr] = acc[n][i];
    }
}

__global__ __launch_bounds__(256) void score_dw_sum_kernel(const float* __restrict__ pw, size_t n,
                                                           int slices, float* __restrict__ d_w) {
  const size_t i = ((size_t)blockIdx.x * 256 + threadIdx.x) * 4;
  if (i >= n) return;
  f32x4 v = *reinterpret_cast<const f32x4*>(pw + i);
  for (int s = 1; s < slices; ++s) v += *reinterpret_cast<const f32x4*>(pw + s * n + i);
  *reinterpret_cast<f32x4*>(d_w + i) = v;
}

static void sum_slices(const ScoreGradArgs& a, int slices, hipStream_t s) {
  const size_t n = (size_t)a.sh.E * a.sh.d;
  score_dw_sum_kernel<<<(unsigned)((n / 4 + 255) / 256), 256, 0, s>>>(a.pw, n, slices, a.d_w);
}

static void products_f32(const ScoreGradArgs& a, hipStream_t s) {
  const ScoreShape& h = a.sh;
  const int pitch = dl_pitch(h.E);
  if (a.d_x)
    score_dx_kernel<<<dim3((h.T + 15) / 16, (h.d + 255) / 256), 256, 0, s>>>(
        a.dl, pitch, static_cast<const float*>(a.w), h.T, h.d, h.E, static_cast<float*>(a.d_x));
  if (a.d_w) {
    const int slices = score_grad_slices(h);
    score_dw_kernel<<<dim3((h.E + 15) / 16, (h.d + 255) / 256, slices), 256, 0, s>>>(
        a.dl, pitch, static_cast<const float*>(a.x), h.T, h.d, h.E, slices, slices > 1 ? a.pw : a.d_w);
    if (slices > 1) sum_slices(a, slices, s);
  }
}

template <int NE>
static void launch_dx(const ScoreGradArgs& a, hipStream_t s) {
  const ScoreShape& h = a.sh;
  const int cols = (h.d + kDxCols - 1) / kDxCols, tiles = (h.T + kDxRows - 1) / kDxRows;
  const int groups = std::min(std::max(1, 256 / cols), tiles);   // one block per CU
  score_dx_bf16_kernel<NE><<<cols * groups, 512, 0, s>>>(
      a.dl, dl_pitch(h.E), static_cast<const uint16_t*>(a.w), h.T, h.d, h.E, groups, static_cast<uint16_t*>(a.d_x));
}

static void products_bf16(const ScoreGradArgs& a, hipStream_t s) {
  const ScoreShape& h = a.sh;
  if (a.d_x) {
    if (h.E <= 64) launch_dx<64>(a, s);
    else if (h.E <= 128) launch_dx<128>(a, s);
    else if (h.E <= 192) launch_dx<192>(a, s);
    else launch_dx<256>(a, s);
  }
  if (a.d_w) {
    const int slices = score_grad_slices(h), cols = (h.d + kGradCols - 1) / kGradCols;
    float* out = slices > 1 ? a.pw : a.d_w;
    const uint16_t* x = static_cast<const uint16_t*>(a.x);
    if (h.E <= 64)
      score_dw_bf16_kernel<1><<<dim3(slices, cols, 1), 256, 0, s>>>(a.dl, dl_pitch(h.E), x, h.T, h.d, h.E, slices, out);
    else
      score_dw_bf16_kernel<2><<<dim3(slices, cols, (h.E + 127) / 128), 256, 0, s>>>(a.dl, dl_pitch(h.E), x, h.T, h.d, h.E,
                                                                                 slices, out);
    if (slices > 1) sum_slices(a, slices, s);
  }
}

template <int PER>                                     // 64 PER: dl_pitch(E)
static void launch_dlogits(const ScoreGradArgs& a, int blocks, hipStream_t s) {
  const bool big = grad_tile(a.sh.T) == 64;
  if (a.sigmoid && big) score_dlogits_kernel<PER, 64, true><<<blocks, 1024, 0, s>>>(a);
  else if (a.sigmoid) score_dlogits_kernel<PER, 16, true><<<blocks, 256, 0, s>>>(a);
  else if (big) score_dlogits_kernel<PER, 64, false><<<blocks, 1024, 0, s>>>(a);
  else score_dlogits_kernel<PER, 16, false><<<blocks, 256, 0, s>>>(a);
}

hipError_t launch_score_grad(const ScoreGradArgs& a, hipStream_t s) {
  const ScoreShape& h = a.sh;
  const int nb = grad_blocks(h.T);
  if (h.E <= 64) launch_dlogits<1>(a, nb, s);
  else if (h.E <= 128) launch_dlogits<2>(a, nb, s);
  else launch_dlogits<4>(a, nb, s);
  if (a.d_b) score_db_kernel<<<(h.E + 3) / 4, 256, 0, s>>>(a.pb, nb, h.E, a.d_b);
  if (h.bf16) products_bf16(a, s);
  else products_f32(a, s);
  return hipGetLastError();
}

}  // namespace moe
