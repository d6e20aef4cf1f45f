// The scored router on gfx950: logits on MFMA, then scores, groups, top-k and
// weights, one wave per token, and the sums over tokens that the losses need.
//
// Web page "Mixture of Experts: Scaling Parameters Without Scaling Compute",
// sections "The MoE layer" (router, top-k, renormalisation) and "The central
// problem: load balancing" (balance loss, z-loss, selection-only bias), with
// sigmoid scores and group-limited selection added.
#include <algorithm>

#include "device_common.h"
#include "score.h"

namespace moe {

constexpr int kPartWaves = 4;       // waves of a logits block, 16 experts each

int score_parts(const ScoreShape& s) {
  // Enough waves to cover the chip twice (512 blocks), no part under 128 of d.
  const long blocks = (long)((s.T + 15) / 16) * ((s.E + 63) / 64);
  const long most = std::min(32L, s.d / 128L);
  return (int)std::max(1L, std::min(most, 512 / blocks));
}

// Few tokens per block keep every CU busy; many blocks would cost the reduction.
int score_finish_blocks(int T) { return std::max(1, std::min(256, (T + 3) / 4)); }

// Partial logits: wave w of block (t-tile, e-tile, part) multiplies 16 tokens by
// 16 experts over its part of d, operands straight from memory to registers.
template <typename T>
__global__ __launch_bounds__(256) void score_logits_kernel(const T* __restrict__ x,
                                                           const T* __restrict__ w, int tokens,
                                                           int d, int E, int parts,
                                                           float* __restrict__ part) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int fr = lane & 15, fc = lane >> 4;
  const int t0 = blockIdx.x * 16, e0 = blockIdx.y * 64 + wave * 16, p = blockIdx.z;
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

__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v = max(v, (uint32_t)__shfl_xor((int)v, o));
  return v;
}
__device__ __forceinline__ float wave_max_f(float v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor(v, o));
  return v;
}
__device__ __forceinline__ float wave_sum_f(float v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  return v;
}

// One wave per token; lane l holds experts l, l + 64, ... (PER of them).
// TRAIN: also the partial sums over this block's tokens.
template <int PER, bool TRAIN>
__global__ __launch_bounds__(256) void score_finish_kernel(ScoreArgs a, int parts) {
  __shared__ float sel_lds[4][64 * PER];
  __shared__ double sum_p[4][64 * PER];
  __shared__ int sum_l[4][64 * PER];
  __shared__ double sum_z[4];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int E = a.sh.E, T = a.sh.T, k = a.sh.k, G = a.groups;
  const int gs = E / G;
  int shift = 0;                                   // lanes per group: 2^shift
  while ((G << (shift + 1)) <= 64) ++shift;
  const int P = 1 << shift;
  int gbit[PER];                                   // lane that knows whether j's group stays
  float bias[PER], bsel[PER];
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const int e = j * 64 + lane;
    gbit[j] = e < E ? (e / gs) << shift : 0;
    bias[j] = (a.b_router && e < E) ? a.b_router[e] : 0.f;
    bsel[j] = (a.b_select && e < E) ? a.b_select[e] : 0.f;
  }
  double pq[PER], pz = 0.0;
  int pl[PER];
#pragma unroll
  for (int j = 0; j < PER; ++j) pq[j] = 0.0, pl[j] = 0;

  for (int t = blockIdx.x * 4 + wave; t < T; t += gridDim.x * 4) {
    float l[PER], s[PER];
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const int e = j * 64 + lane;
      l[j] = 0.f;
      if (e < E)
        for (int p = 0; p < parts; ++p) l[j] += a.part[((size_t)p * T + t) * E + e];
      l[j] = e < E ? l[j] + bias[j] : -INFINITY;
      if (a.logits && e < E) a.logits[(size_t)t * E + e] = l[j];
    }
    float m = l[0], tot = 0.f;
    if (TRAIN || !a.sigmoid) {
#pragma unroll
      for (int j = 1; j < PER; ++j) m = fmaxf(m, l[j]);
      m = wave_max_f(m);
      if (m == -INFINITY) m = 0.f;                 // every logit -inf: all scores 0
#pragma unroll
      for (int j = 0; j < PER; ++j) {
        s[j] = j * 64 + lane < E ? expf(l[j] - m) : 0.f;
        tot += s[j];
      }
      tot = wave_sum_f(tot);
    }
    if (TRAIN && a.z_loss) {
      const double lse = (double)m + (double)logf(tot);
      pz += lse * lse;
    }
    if (a.sigmoid) {
#pragma unroll
      for (int j = 0; j < PER; ++j) s[j] = j * 64 + lane < E ? 1.f / (1.f + expf(-l[j])) : 0.f;
    } else {
#pragma unroll
      for (int j = 0; j < PER; ++j) s[j] /= tot > 0.f ? tot : 1.f;
    }
    if (TRAIN) {
      float q = 1.f;
      if (a.sigmoid) {
        q = 0.f;
#pragma unroll
        for (int j = 0; j < PER; ++j) q += s[j];
        q = fmaxf(wave_sum_f(q), 1e-20f);          // every score underflowed: q = 0
      }
#pragma unroll
      for (int j = 0; j < PER; ++j) pq[j] += (double)(s[j] / q);
    }

    uint32_t key[PER];
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const float v = s[j] + bsel[j];
      key[j] = j * 64 + lane < E ? order_key(v) : 0u;
      if (G > 1) sel_lds[wave][j * 64 + lane] = v == v ? v : -INFINITY;
    }
    if (G > 1) {
      // Lanes [g P, (g + 1) P) find the best two of group g.
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
      __builtin_amdgcn_wave_barrier();
      float b0 = -INFINITY, b1 = -INFINITY;
      const int g = lane >> shift;
      if (g < G)
        for (int i = lane & (P - 1); i < gs; i += P) {
          const float v = sel_lds[wave][g * gs + i];
          b1 = fmaxf(b1, fminf(b0, v));
          b0 = fmaxf(b0, v);
        }
      __builtin_amdgcn_wave_barrier();
      for (int o = 1; o < P; o <<= 1) {
        const float c0 = __shfl_xor(b0, o), c1 = __shfl_xor(b1, o);
        b1 = fmaxf(fmaxf(b1, c1), fminf(b0, c0));
        b0 = fmaxf(b0, c0);
      }
      const uint32_t gk = g < G ? order_key(a.group_top == 2 ? b0 + b1 : b0) : 0u;
      int rank = 0;
      for (int h = 0; h < G; ++h) {
        const uint32_t hk = (uint32_t)__shfl((int)gk, h << shift);
        rank += hk > gk || (hk == gk && h < g);
      }
      const uint64_t stay = __ballot(g < G && rank < a.top_groups);
#pragma unroll
      for (int j = 0; j < PER; ++j)
        if (!((stay >> gbit[j]) & 1)) key[j] = 0u;
    }

    // Top-k: the wave's best value, then the lowest expert that has it.
    float my_r = 0.f, total = 0.f;
    int my_e = 0;
    for (int i = 0; i < k; ++i) {
      uint32_t best = key[0];
#pragma unroll
      for (int j = 1; j < PER; ++j) best = max(best, key[j]);
      best = wave_max_u32(best);
      int e = -1;
      float r = 0.f;
#pragma unroll
      for (int j = 0; j < PER; ++j) {
        if (e < 0) {
          const uint64_t hit = __ballot(key[j] == best);
          if (hit) {
            const int at = __ffsll((unsigned long long)hit) - 1;
            e = j * 64 + at;
            r = __shfl(s[j], at);
            if (lane == at) {
              key[j] = 0u;
              if (TRAIN) ++pl[j];
            }
          }
        }
      }
      total += r;
      if (lane == i) my_r = r, my_e = e;
    }
    if (lane < k) {
      a.topk_idx[(size_t)t * k + lane] = my_e;
      a.topk_w[(size_t)t * k + lane] = a.renorm ? a.scale * (my_r / (total + 1e-20f)) : a.scale * my_r;
    }
  }

  if constexpr (TRAIN) {
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      sum_p[wave][j * 64 + lane] = pq[j];
      sum_l[wave][j * 64 + lane] = pl[j];
    }
    if (lane == 0) sum_z[wave] = pz;
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += 256) {
      a.psum[(size_t)blockIdx.x * E + e] = sum_p[0][e] + sum_p[1][e] + sum_p[2][e] + sum_p[3][e];
      a.pload[(size_t)blockIdx.x * E + e] = sum_l[0][e] + sum_l[1][e] + sum_l[2][e] + sum_l[3][e];
    }
    if (threadIdx.x == 0) a.pz[blockIdx.x] = sum_z[0] + sum_z[1] + sum_z[2] + sum_z[3];
  }
}

// The sums over blocks, in a fixed order, and what follows from them.  1024
// threads: expert tid % 256, quarter tid / 256 of the blocks.
__global__ __launch_bounds__(1024) void score_reduce_kernel(ScoreArgs a, int blocks) {
  __shared__ double sp[4][kScoreMaxExperts];
  __shared__ int sl[4][kScoreMaxExperts];
  __shared__ double sx[kScoreMaxExperts], sz[kScoreMaxExperts];
  const int e = threadIdx.x & 255, q = threadIdx.x >> 8, E = a.sh.E;
  double p = 0.0;
  int n = 0;
  if (e < E)
    for (int b = q; b < blocks; b += 4) {
      p += a.psum[(size_t)b * E + e];
      n += a.pload[(size_t)b * E + e];
    }
  sp[q][e] = p;
  sl[q][e] = n;
  if (q == 0) sz[e] = e < blocks ? a.pz[e] : 0.0;   // at most 256 blocks
  __syncthreads();
  if (q == 0) {
    double v = 0.0;
    if (e < E) {
      const double mean = (sp[0][e] + sp[1][e] + sp[2][e] + sp[3][e]) / a.sh.T;
      const int load = sl[0][e] + sl[1][e] + sl[2][e] + sl[3][e];
      if (a.prob_mean) a.prob_mean[e] = (float)mean;
      if (a.load) a.load[e] = load;
      v = mean * load;
    }
    sx[e] = v;
  }
  for (int o = 128; o > 0; o >>= 1) {
    __syncthreads();
    if ((int)threadIdx.x < o) {
      sx[threadIdx.x] += sx[threadIdx.x + o];
      sz[threadIdx.x] += sz[threadIdx.x + o];
    }
  }
  if (threadIdx.x == 0) {
    if (a.aux) *a.aux = (float)(sx[0] * E / ((double)a.sh.T * a.sh.k));
    if (a.z_loss) *a.z_loss = (float)(sz[0] / a.sh.T);
  }
}

hipError_t launch_score(const ScoreArgs& a, hipStream_t s) {
  const ScoreShape& h = a.sh;
  const int parts = score_parts(h), nb = score_finish_blocks(h.T);
  const dim3 grid((h.T + 15) / 16, (h.E + 63) / 64, parts);
  if (h.bf16)
    score_logits_kernel<uint16_t><<<grid, 256, 0, s>>>(static_cast<const uint16_t*>(a.x),
                                                      static_cast<const uint16_t*>(a.w), h.T, h.d,
                                                      h.E, parts, a.part);
  else
    score_logits_kernel<float><<<grid, 256, 0, s>>>(static_cast<const float*>(a.x),
                                                   static_cast<const float*>(a.w), h.T, h.d, h.E,
                                                   parts, a.part);
  const bool train = a.load || a.prob_mean || a.aux || a.z_loss;
  auto finish = [&](auto per) {
    constexpr int PER = decltype(per)::value;
    if (train)
      score_finish_kernel<PER, true><<<nb, 256, 0, s>>>(a, parts);
    else
      score_finish_kernel<PER, false><<<nb, 256, 0, s>>>(a, parts);
  };
  if (h.E <= 64) finish(std::integral_constant<int, 1>{});
  else if (h.E <= 128) finish(std::integral_constant<int, 2>{});
  else finish(std::integral_constant<int, 4>{});
  if (train) score_reduce_kernel<<<1, 1024, 0, s>>>(a, nb);
  return hipGetLastError();
}

}  // namespace moe
