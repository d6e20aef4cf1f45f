// Layer norm over rows of d values, with the residual add before it, and its gradients.
//
//   h = x + add (rounded to x's type, the residual stream)
//   mean = sum h / d,  rstd = 1 / sqrt(sum (h - mean)^2 / d + eps)
//   y = (h - mean) rstd w + b
// Backward, with hat = (h - mean) rstd and g = dy w:
//   d_x = rstd (g - mean(g) - hat mean(g hat)) + d_x_out
//   d_w = sum over rows of dy hat,  d_b = sum over rows of dy
//
// Memory bounds both.  A group of G threads has a row in registers (8 NV values a thread), so
// it is read once and the squares are those of the differences from the mean; the groups take
// rows in turn, and their threads keep the same columns, so weight and bias stay in
// registers, and so do the column sums of the backward pass.  Those are written once a block
// and added up, in order, by a second kernel.  Everything is summed in fp32.
//
// 16384 x 4096 bf16, fp32 add: 124 us, 5.4 TB/s; gradients with d_x_out 106 us, 5.0 TB/s, of which
// the second kernel takes 4.9; fp32 208 and 206 us, 5.2 TB/s.  One row of 4096 is 3.4 us.
// 1024 threads have 128 registers each: past 8192 columns some of the gradients' spill (10 to 130), past 16384 the
// forward's too (50 to 240) and most of the gradients' (400 to 460), and go through the caches.  2000 x 32768 bf16
// 183 and 556 us, 1000 x 32768 fp32 183 and 432; 132 and 106, 106 and 106 by bytes at a copy's rate.
#include <algorithm>

#include "device_common.h"
#include "norm.h"

namespace moe {

// ---- eight values at a time --------------------------------------------------------------
__device__ __forceinline__ void load8(const uint16_t* p, float (&v)[8]) {
  const u32x4 u = ld16(p);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(u[i] << 16);
    v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const f32x4 a = *reinterpret_cast<const f32x4*>(p), b = *reinterpret_cast<const f32x4*>(p + 4);
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = a[i], v[4 + i] = b[i];
}
__device__ __forceinline__ void store8(uint16_t* p, const float (&v)[8]) {
  u32x4 u;
#pragma unroll
  for (int i = 0; i < 4; ++i) u[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
  st16(p, u);
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  *reinterpret_cast<f32x4*>(p) = (f32x4){v[0], v[1], v[2], v[3]};
  *reinterpret_cast<f32x4*>(p + 4) = (f32x4){v[4], v[5], v[6], v[7]};
}
__device__ __forceinline__ float load1(const uint16_t* p) { return bf16_to_f32(*p); }
__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ void store1(uint16_t* p, float v) { *p = (uint16_t)pack_bf16x2(v, 0.f); }
__device__ __forceinline__ void store1(float* p, float v) { *p = v; }
// The value that is stored.
__device__ __forceinline__ float stored(float v, uint16_t) { return __uint_as_float(pack_bf16x2(v, 0.f) << 16); }
__device__ __forceinline__ float stored(float v, float) { return v; }

// Which columns thread t of a group of G holds: VEC, eight neighbours per 8 G columns (rows
// of whole 16-byte pieces); else every G-th, so that odd widths and strides still read whole
// lines.  Columns at and past d hold 0.
template <int G, int NV, bool VEC>
struct Columns {
  // Odd widths: every load under way before the first is used, while registers last (3000 x 4095 bf16 35 us
  // against 52 behind branches; 3000 x 14999 in 1024 threads 397 against 175).
  static constexpr bool kWhole = G <= 512;
  static __device__ __forceinline__ int at(int t, int v, int j) {
    return VEC ? (v * G + t) * 8 + j : (v * 8 + j) * G + t;
  }
  template <typename T>
  static __device__ __forceinline__ void load(const T* row, int t, int d, float (&x)[NV][8]) {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      if constexpr (VEC) {
        if (at(t, v, 0) < d) {
          load8(row + at(t, v, 0), x[v]);
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) x[v][j] = 0.f;
        }
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if constexpr (kWhole) x[v][j] = load1(row + min(at(t, v, j), d - 1));
          else x[v][j] = at(t, v, j) < d ? load1(row + at(t, v, j)) : 0.f;
        }
      }
    }
    if constexpr (!VEC && kWhole)
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int j = 0; j < 8; ++j) x[v][j] = at(t, v, j) < d ? x[v][j] : 0.f;
  }
  template <typename T>
  static __device__ __forceinline__ void store(T* row, int t, int d, const float (&x)[NV][8]) {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      if constexpr (VEC) {
        if (at(t, v, 0) < d) store8(row + at(t, v, 0), x[v]);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (at(t, v, j) < d) store1(row + at(t, v, j), x[v][j]);
      }
    }
  }
  // weight or bias, of either type, or `none` where there is none
  static __device__ __forceinline__ void load_param(const void* p, bool bf16, float none, int t, int d,
                                                    float (&x)[NV][8]) {
    if (!p) {
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int j = 0; j < 8; ++j) x[v][j] = none;
    } else if (bf16) {
      load(static_cast<const uint16_t*>(p), t, d, x);
    } else {
      load(static_cast<const float*>(p), t, d, x);
    }
  }
};

constexpr int waves_of(int G) { return G < 64 ? 1 : G / 64; }

// Sums of N values over a group, returned to all its threads.  Groups wider than a wave
// exchange through `red`; calls alternate its halves, so one barrier each is enough.
template <int G, int N>
struct GroupSum {
  static constexpr int kW = waves_of(G);
  float (*red)[N][kW];
  int half = 0;
  __device__ __forceinline__ void operator()(float (&v)[N]) {
#pragma unroll
    for (int n = 0; n < N; ++n) v[n] = G < 64 ? lanes_sum<(G < 64 ? G : 64)>(v[n]) : wave_sum_f(v[n]);
    if constexpr (kW > 1) {
      if ((threadIdx.x & 63) == 0)
#pragma unroll
        for (int n = 0; n < N; ++n) red[half][n][threadIdx.x >> 6] = v[n];
      __syncthreads();
#pragma unroll
      for (int n = 0; n < N; ++n) {
        float s = red[half][n][0];
#pragma unroll
        for (int w = 1; w < kW; ++w) s += red[half][n][w];
        v[n] = s;
      }
      half ^= 1;
    }
  }
};

constexpr int block_of(int G) { return G < 256 ? 256 : G; }

template <typename T, int G, int NV, bool VEC>
__global__ __launch_bounds__(block_of(G)) void norm_kernel(NormArgs a) {
  using C = Columns<G, NV, VEC>;
  constexpr int kGroups = block_of(G) / G;
  __shared__ float red[2][1][waves_of(G)];
  GroupSum<G, 1> sum{red};
  const int t = threadIdx.x % G, d = a.sh.d;
  const float inv = 1.f / d;
  float w[NV][8], b[NV][8];
  C::load_param(a.weight, a.sh.w_bf16, 1.f, t, d, w);
  C::load_param(a.bias, a.sh.w_bf16, 0.f, t, d, b);
  for (int64_t row = (int64_t)blockIdx.x * kGroups + threadIdx.x / G; row < a.sh.rows;
       row += (int64_t)gridDim.x * kGroups) {
    float x[NV][8];
    C::load(static_cast<const T*>(a.x.p) + row * a.x.stride, t, d, x);
    if (a.add.p) {
      float r[NV][8];
      if (a.sh.add_bf16) C::load(static_cast<const uint16_t*>(a.add.p) + row * a.add.stride, t, d, r);
      else C::load(static_cast<const float*>(a.add.p) + row * a.add.stride, t, d, r);
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int j = 0; j < 8; ++j) x[v][j] = stored(x[v][j] + r[v][j], T());
    }
    if (a.x_out.p) C::store(static_cast<T*>(a.x_out.p) + row * a.x_out.stride, t, d, x);
    float s[1] = {0.f};
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int j = 0; j < 8; ++j) s[0] += x[v][j];
    sum(s);
    const float mean = s[0] * inv;
    s[0] = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        x[v][j] -= mean;
        if (C::at(t, v, VEC ? 0 : j) < d) s[0] = fmaf(x[v][j], x[v][j], s[0]);
      }
    sum(s);
    const float rstd = 1.f / sqrtf(fmaf(s[0], inv, a.sh.eps));
    if (t == 0) {
      if (a.mean) a.mean[row] = mean;
      if (a.rstd) a.rstd[row] = rstd;
    }
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int j = 0; j < 8; ++j) x[v][j] = fmaf(x[v][j] * rstd, w[v][j], b[v][j]);
    C::store(static_cast<T*>(a.y.p) + row * a.y.stride, t, d, x);
  }
}

// A row's values as they lie in memory, so that the next row can be under way in few registers.
template <typename T, int G, int NV, bool VEC>
struct RawRow {
  using C = Columns<G, NV, VEC>;
  static constexpr int kWords = VEC ? sizeof(T) / 2 : 1;
  u32x4 v[NV][kWords];                               // VEC: 8 values
  float s[VEC ? 1 : NV][8];
  __device__ __forceinline__ void load(const T* row, int t, int d) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if constexpr (VEC) {
#pragma unroll
        for (int w = 0; w < kWords; ++w)
          v[i][w] = ld16(row + min(C::at(t, i, 0), d - 8) + w * (16 / sizeof(T)));
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) s[i][j] = load1(row + min(C::at(t, i, j), d - 1));
      }
    }
  }
  // Columns at and past d are 0.
  __device__ __forceinline__ void get(int t, int d, float (&x)[NV][8]) const {
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float f;
        if constexpr (!VEC) f = s[i][j];
        else if constexpr (sizeof(T) == 4) f = __uint_as_float(v[i][j / 4][j % 4]);
        else f = __uint_as_float(j % 2 ? v[i][0][j / 2] & 0xffff0000u : v[i][0][j / 2] << 16);
        x[i][j] = C::at(t, i, VEC ? 0 : j) < d ? f : 0.f;
      }
  }
};

template <typename T, int G, int NV, bool VEC>
__global__ __launch_bounds__(block_of(G)) void norm_grad_kernel(NormGradArgs a) {
  using C = Columns<G, NV, VEC>;
  constexpr int kGroups = block_of(G) / G;
  __shared__ float red[2][2][waves_of(G)];
  GroupSum<G, 2> sum{red};
  const int t = threadIdx.x % G, d = a.sh.d;
  const int64_t group = (int64_t)blockIdx.x * kGroups + threadIdx.x / G, step = (int64_t)gridDim.x * kGroups;
  const float inv = 1.f / d;
  float w[NV][8], dw[NV][8] = {}, db[NV][8] = {};
  C::load_param(a.weight, a.sh.w_bf16, 1.f, t, d, w);
  RawRow<T, G, NV, VEC> nx, ng, nr;
  float next_mean, next_rstd;
  const bool through = a.d_x_out.p;
  auto fetch = [&](int64_t row) {                    // past the end: the last row again, not used
    row = row < a.sh.rows ? row : a.sh.rows - 1;
    ng.load(static_cast<const T*>(a.dy.p) + row * a.dy.stride, t, d);
    nx.load(static_cast<const T*>(a.x.p) + row * a.x.stride, t, d);
    if (through) nr.load(static_cast<const T*>(a.d_x_out.p) + row * a.d_x_out.stride, t, d);
    next_mean = a.mean[row];
    next_rstd = a.rstd[row];
  };
  constexpr bool kAhead = VEC && G <= 512;           // else the next row's registers would spill
  if (kAhead) fetch(group);
  for (int64_t row = group; row < a.sh.rows; row += step) {
    if (!kAhead) fetch(row);
    float x[NV][8], g[NV][8], r[NV][8];
    ng.get(t, d, g);
    nx.get(t, d, x);
    if (through) {
      nr.get(t, d, r);
    } else {
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int j = 0; j < 8; ++j) r[v][j] = 0.f;
    }
    const float mean = next_mean, rstd = next_rstd;
    if (kAhead) fetch(row + step);
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        // past d: (0 - mean) rstd may be anything, its dy is 0
        x[v][j] = C::at(t, v, VEC ? 0 : j) < d ? (x[v][j] - mean) * rstd : 0.f;
        dw[v][j] = fmaf(g[v][j], x[v][j], dw[v][j]);
        db[v][j] += g[v][j];
        g[v][j] *= w[v][j];
        s[0] += g[v][j];
        s[1] = fmaf(g[v][j], x[v][j], s[1]);
      }
    if (a.d_x.p) {
      sum(s);
      s[0] *= inv;
      s[1] *= inv;
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int j = 0; j < 8; ++j) r[v][j] = fmaf(rstd, g[v][j] - fmaf(x[v][j], s[1], s[0]), r[v][j]);
      C::store(static_cast<T*>(a.d_x.p) + row * a.d_x.stride, t, d, r);
    }
  }
  // One row of partial sums a block: its groups' added up, by lanes, then by waves.
  float* part = a.part + (size_t)blockIdx.x * 2 * d;
  if constexpr (kGroups > 1) {
    __shared__ float all[4][2][8 * G * NV];
    if (!a.d_weight && !a.d_bias) return;
    const int wave = threadIdx.x >> 6;
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
#pragma unroll
        for (int o = G; o < 64; o <<= 1) {
          dw[v][j] += __shfl_xor(dw[v][j], o);
          db[v][j] += __shfl_xor(db[v][j], o);
        }
        if ((threadIdx.x & 63) < G) {
          all[wave][0][C::at(t, v, j)] = dw[v][j];
          all[wave][1][C::at(t, v, j)] = db[v][j];
        }
      }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * d; i += 256) {
      const int b = i >= d, c = b ? i - d : i;
      part[i] = (all[0][b][c] + all[1][b][c]) + (all[2][b][c] + all[3][b][c]);
    }
  } else {
    if (a.d_weight) C::store(part, t, d, dw);
    if (a.d_bias) C::store(part + d, t, d, db);
  }
}

// Column sums of the blocks' partial rows [groups][2 d]: 64 columns a block here, 16 waves a
// sixteenth of the rows each.
__global__ __launch_bounds__(1024) void norm_sum_kernel(const float* __restrict__ part, int groups, int d,
                                                        float* __restrict__ d_weight, float* __restrict__ d_bias) {
  __shared__ float acc[16][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int c = blockIdx.x * 64 + lane;
  float* out = c < d ? d_weight : d_bias;
  const bool live = c < 2 * d && out;
  float s = 0.f;
  if (live)
#pragma unroll 8
    for (int g = wave; g < groups; g += 16) s += part[(size_t)g * 2 * d + c];
  acc[wave][lane] = s;
  __syncthreads();
  if (wave == 0 && live) {
#pragma unroll
    for (int w = 1; w < 16; ++w) s += acc[w][lane];
    out[c < d ? c : c - d] = s;
  }
}

// ---- launches ----------------------------------------------------------------------------
// Threads of a row: as few as hold it with 8 values each up to a wave (64 values in 64 lanes took
// twice as long), then 16.
static int group_of(int d) {
  return d <= 64 ? 8 : d <= 128 ? 16 : d <= 256 ? 32 : d <= 1024 ? 64 : d <= 4096 ? 256 : d <= 8192 ? 512 : 1024;
}
static int groups_per_block(int d) { return block_of(group_of(d)) / group_of(d); }

static int blocks_for(const NormShape& s, int most) {
  const int per = groups_per_block(s.d);
  return (int)std::min<int64_t>((s.rows + per - 1) / per, most);
}
// Four rows a group at least, or the sums of their sums take longer than they; at most 512 blocks
// (256: 16384 x 2048 85 us against 63).  Past 4096 columns two rows (200 x 16384 fp32 35 us, with four 48)
// and 256 blocks (2048 x 8192 34 us against 41).
static int grad_blocks(const NormShape& s) {
  const int64_t rows = (s.d > 4096 ? 2 : 4) * groups_per_block(s.d);
  return (int)std::min<int64_t>((s.rows + rows - 1) / rows, s.d > 4096 ? 256 : 512);
}

size_t norm_grad_part_bytes(const NormShape& s) { return (size_t)grad_blocks(s) * 2 * s.d * 4; }

// Rows of whole 16-byte pieces of eight values.
template <typename P>
static bool whole(const Rows<P>& r, int64_t rows, bool bf16) {
  return !r.p || rows <= 1 || r.stride % (bf16 ? 8 : 4) == 0;
}

template <typename T, typename F>
static void for_width(int d, bool vec, F f) {
  auto with = [&](auto g, auto nv) {
    if (vec) f(g, nv, std::true_type());
    else f(g, nv, std::false_type());
  };
  using std::integral_constant;
  if (d <= 64) with(integral_constant<int, 8>(), integral_constant<int, 1>());
  else if (d <= 128) with(integral_constant<int, 16>(), integral_constant<int, 1>());
  else if (d <= 256) with(integral_constant<int, 32>(), integral_constant<int, 1>());
  else if (d <= 512) with(integral_constant<int, 64>(), integral_constant<int, 1>());
  else if (d <= 1024) with(integral_constant<int, 64>(), integral_constant<int, 2>());
  else if (d <= 2048) with(integral_constant<int, 256>(), integral_constant<int, 1>());
  else if (d <= 4096) with(integral_constant<int, 256>(), integral_constant<int, 2>());
  else if (d <= 8192) with(integral_constant<int, 512>(), integral_constant<int, 2>());
  else if (d <= 16384) with(integral_constant<int, 1024>(), integral_constant<int, 2>());
  else with(integral_constant<int, 1024>(), integral_constant<int, 4>());
}

template <typename T>
static void run_norm(const NormArgs& a, hipStream_t s) {
  const NormShape& n = a.sh;
  const bool vec = n.d % 8 == 0 && whole(a.x, n.rows, n.bf16) && whole(a.add, n.rows, n.add_bf16) &&
                   whole(a.x_out, n.rows, n.bf16) && whole(a.y, n.rows, n.bf16);
  const int blocks = blocks_for(n, 2048);
  for_width<T>(n.d, vec, [&](auto g, auto nv, auto v) {
    constexpr int G = decltype(g)::value;
    norm_kernel<T, G, decltype(nv)::value, decltype(v)::value><<<blocks, block_of(G), 0, s>>>(a);
  });
}

hipError_t launch_norm(const NormArgs& a, hipStream_t s) {
  if (a.sh.rows == 0) return hipSuccess;
  if (a.sh.bf16) run_norm<uint16_t>(a, s);
  else run_norm<float>(a, s);
  return hipGetLastError();
}

template <typename T>
static void run_grad(const NormGradArgs& a, int blocks, hipStream_t s) {
  const NormShape& n = a.sh;
  const bool vec = n.d % 8 == 0 && whole(a.x, n.rows, n.bf16) && whole(a.dy, n.rows, n.bf16) &&
                   whole(a.d_x_out, n.rows, n.bf16) && whole(a.d_x, n.rows, n.bf16);
  for_width<T>(n.d, vec, [&](auto g, auto nv, auto v) {
    constexpr int G = decltype(g)::value;
    norm_grad_kernel<T, G, decltype(nv)::value, decltype(v)::value><<<blocks, block_of(G), 0, s>>>(a);
  });
}

hipError_t launch_norm_grad(const NormGradArgs& a, hipStream_t s) {
  const int blocks = grad_blocks(a.sh);
  if (blocks > 0) {
    if (a.sh.bf16) run_grad<uint16_t>(a, blocks, s);
    else run_grad<float>(a, blocks, s);
    if (hipError_t e = hipGetLastError()) return e;
  }
  if (a.d_weight || a.d_bias)                        // no rows: zeros
    norm_sum_kernel<<<(2 * a.sh.d + 63) / 64, 1024, 0, s>>>(a.part, blocks, a.sh.d,
                                                             a.d_weight, a.d_bias);
  return hipGetLastError();
}

}  // namespace moe
