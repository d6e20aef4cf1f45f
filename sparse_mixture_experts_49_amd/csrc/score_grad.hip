// Gradients of the scored router on gfx950.
//
// For each token, with g = d topk_w, chosen scores r_j = s[idx_j], S = sum r + 1e-20:
//   dr_j = scale g_j, or renormalised (scale g_j - sum_i g_i w_i) / S
//   dq_e = d_aux E load_e / (T k) / T          (q = s / sum s; load is a constant)
//   softmax: ds = dr + dq;                       dl = s (ds - sum ds s)
//   sigmoid: ds = dr + (dq - sum dq q) / sum s;  dl = ds s (1 - s)
//   dl += d_z (2 / T) lse softmax(l)
// and d_b = sum_t dl, d_x = dl W_r, d_W = dl^T x.
#include <algorithm>

#include "device_common.h"
#include "score.h"

namespace moe {

int score_grad_slices(const ScoreShape& s) {
  // d_w_router tiles of 16 experts x 64 columns per wave; slices of at least 64
  // tokens until 1024 waves run.
  const long tiles = (long)((s.E + 15) / 16) * (s.d / 64);
  return (int)std::max(1L, std::min({16L, (long)(s.T + 63) / 64, 2048 / tiles}));
}

__device__ __forceinline__ float wsum(float v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  return v;
}

// One wave per token; lane l holds experts l, l + 64, ...
template <int PER>
__global__ __launch_bounds__(256) void score_dlogits_kernel(ScoreGradArgs a) {
  __shared__ double sum_b[4][64 * PER];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int E = a.sh.E, T = a.sh.T, k = a.sh.k;
  float dq[PER];
  const float aux = a.d_aux ? *a.d_aux : 0.f, z = a.d_z ? *a.d_z : 0.f;
  double pb[PER];
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const int e = j * 64 + lane;
    dq[j] = (a.d_aux && e < E)
                ? (float)((double)aux * E * a.load[e] / ((double)T * k) / T)
                : 0.f;
    pb[j] = 0.0;
  }
  for (int t = blockIdx.x * 4 + wave; t < T; t += gridDim.x * 4) {
    float l[PER], p[PER], s[PER];
    float m = -INFINITY;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const int e = j * 64 + lane;
      l[j] = e < E ? a.logits[(size_t)t * E + e] : -INFINITY;
      m = fmaxf(m, l[j]);
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor(m, o));
    if (m == -INFINITY) m = 0.f;
    float tot = 0.f;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      p[j] = j * 64 + lane < E ? expf(l[j] - m) : 0.f;
      tot += p[j];
    }
    tot = wsum(tot);
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      p[j] /= tot > 0.f ? tot : 1.f;
      s[j] = !a.sigmoid ? p[j] : j * 64 + lane < E ? 1.f / (1.f + expf(-l[j])) : 0.f;
    }
    // Chosen scores and the gradients of the raw weights.
    int idx[8];
    float g[8], S = 1e-20f, gw = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      idx[i] = i < k ? a.topk_idx[(size_t)t * k + i] : -1;
      if (idx[i] >= E) idx[i] = -1;
      g[i] = (idx[i] >= 0 && a.d_topk_w) ? a.d_topk_w[(size_t)t * k + i] : 0.f;
      float r = 0.f;
#pragma unroll
      for (int j = 0; j < PER; ++j) {
        const float v = __shfl(s[j], idx[i] & 63);
        if (idx[i] >= 0 && (idx[i] >> 6) == j) r = v;
      }
      S += r;
      gw = fmaf(g[i], r, gw);
    }
    float ds[PER];
    float cs = 0.f, cq = 0.f, ss = 0.f;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      float dr = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (idx[i] == j * 64 + lane) dr += a.renorm ? a.scale * (g[i] - gw / S) / S : a.scale * g[i];
      ds[j] = dr;
      ss += s[j];
      cq = fmaf(dq[j], s[j], cq);
    }
    if (a.sigmoid && a.d_aux) {
      ss = fmaxf(wsum(ss), 1e-20f);
      cq = wsum(cq);
#pragma unroll
      for (int j = 0; j < PER; ++j) ds[j] += (dq[j] - cq / ss) / ss;
    } else if (!a.sigmoid) {
#pragma unroll
      for (int j = 0; j < PER; ++j) {
        ds[j] += dq[j];
        cs = fmaf(ds[j], s[j], cs);
      }
      cs = wsum(cs);
    }
    const float zl = a.d_z ? z * 2.f / T * (m + logf(tot)) : 0.f;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const int e = j * 64 + lane;
      float v = a.sigmoid ? ds[j] * s[j] * (1.f - s[j]) : s[j] * (ds[j] - cs);
      v = fmaf(zl, p[j], v);
      if (e < E) {
        a.dl[(size_t)t * E + e] = v;
        if (a.d_logits) a.d_logits[(size_t)t * E + e] = v;
        pb[j] += (double)v;
      }
    }
  }
  if (a.d_b) {
#pragma unroll
    for (int j = 0; j < PER; ++j) sum_b[wave][j * 64 + lane] = pb[j];
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += 256)
      a.pb[(size_t)blockIdx.x * E + e] = sum_b[0][e] + sum_b[1][e] + sum_b[2][e] + sum_b[3][e];
  }
}

__global__ __launch_bounds__(1024) void score_db_kernel(const double* __restrict__ pb, int blocks,
                                                        int E, float* __restrict__ d_b) {
  __shared__ double s[4][kScoreMaxExperts];
  const int e = threadIdx.x & 255, q = threadIdx.x >> 8;
  double p = 0.0;
  if (e < E)
    for (int b = q; b < blocks; b += 4) p += pb[(size_t)b * E + e];
  s[q][e] = p;
  __syncthreads();
  if (q == 0 && e < E) d_b[e] = (float)(s[0][e] + s[1][e] + s[2][e] + s[3][e]);
}

template <typename T>
__device__ __forceinline__ float as_f32(T v) { return Elem<T>::to_f32(v); }

// d_x tile of 16 tokens x 64 columns per wave: k-slot q of MFMA i is expert e0 + 4 i + q.
template <typename T>
__global__ __launch_bounds__(256) void score_dx_kernel(const float* __restrict__ dl,
                                                       const T* __restrict__ w, int tokens, int d,
                                                       int E, T* __restrict__ d_x) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, fr = lane & 15, fc = lane >> 4;
  const int t0 = blockIdx.x * 16, c0 = (blockIdx.y * 4 + wave) * 64;
  if (c0 >= d) return;
  const int t = min(t0 + fr, tokens - 1);
  f32x4 acc[4] = {};
  for (int e0 = 0; e0 < E; e0 += 4) {
    const int e = e0 + fc;
    const float a = e < E ? dl[(size_t)t * E + e] : 0.f;
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      const float b = e < E ? as_f32<T>(w[(size_t)e * d + c0 + n * 16 + fr]) : 0.f;
      acc[n] = mfma_f32(a, b, acc[n]);
    }
  }
#pragma unroll
  for (int n = 0; n < 4; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = t0 + 4 * fc + i;
      if (row >= tokens) continue;
      T* out = d_x + (size_t)row * d + c0 + n * 16 + fr;
      if constexpr (sizeof(T) == 2) *out = f32_to_bf16(acc[n][i]);
      else *out = acc[n][i];
    }
}

// d_w_router tile of 16 experts x 64 columns per wave over one slice of the tokens.
template <typename T>
__global__ __launch_bounds__(256) void score_dw_kernel(const float* __restrict__ dl,
                                                       const T* __restrict__ x, int tokens, int d,
                                                       int E, int slices, float* __restrict__ out) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, fr = lane & 15, fc = lane >> 4;
  const int e0 = blockIdx.x * 16, c0 = (blockIdx.y * 4 + wave) * 64, sl = blockIdx.z;
  if (c0 >= d) return;
  const int ta = (int)((long)sl * tokens / slices), tb = (int)((long)(sl + 1) * tokens / slices);
  const int e = min(e0 + fr, E - 1);
  f32x4 acc[4] = {};
  for (int t0 = ta; t0 < tb; t0 += 4) {
    const int t = t0 + fc;
    const float a = t < tb ? dl[(size_t)t * E + e] : 0.f;
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      const float b = t < tb ? as_f32<T>(x[(size_t)t * d + c0 + n * 16 + fr]) : 0.f;
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

template <typename T>
static void launch_products(const ScoreGradArgs& a, hipStream_t s) {
  const ScoreShape& h = a.sh;
  if (a.d_x)
    score_dx_kernel<T><<<dim3((h.T + 15) / 16, (h.d + 255) / 256), 256, 0, s>>>(
        a.dl, static_cast<const T*>(a.w), h.T, h.d, h.E, static_cast<T*>(a.d_x));
  if (a.d_w) {
    const int slices = score_grad_slices(h);
    score_dw_kernel<T><<<dim3((h.E + 15) / 16, (h.d + 255) / 256, slices), 256, 0, s>>>(
        a.dl, static_cast<const T*>(a.x), h.T, h.d, h.E, slices, slices > 1 ? a.pw : a.d_w);
    if (slices > 1) {
      const size_t n = (size_t)h.E * h.d;
      score_dw_sum_kernel<<<(unsigned)((n / 4 + 255) / 256), 256, 0, s>>>(a.pw, n, slices, a.d_w);
    }
  }
}

hipError_t launch_score_grad(const ScoreGradArgs& a, hipStream_t s) {
  const ScoreShape& h = a.sh;
  const int nb = score_finish_blocks(h.T);
  if (h.E <= 64) score_dlogits_kernel<1><<<nb, 256, 0, s>>>(a);
  else if (h.E <= 128) score_dlogits_kernel<2><<<nb, 256, 0, s>>>(a);
  else score_dlogits_kernel<4><<<nb, 256, 0, s>>>(a);
  if (a.d_b) score_db_kernel<<<1, 1024, 0, s>>>(a.pb, nb, h.E, a.d_b);
  if (h.bf16) launch_products<uint16_t>(a, s);
  else launch_products<float>(a, s);
  return hipGetLastError();
}

}  // namespace moe
