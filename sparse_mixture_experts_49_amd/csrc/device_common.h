// Device helpers shared by the gfx950 kernels of the MoE layer.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace moe {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kWave = 64;

// 16-byte global / LDS vector accesses.
__device__ __forceinline__ u32x4 ld16(const void* p) { return *reinterpret_cast<const u32x4*>(p); }
__device__ __forceinline__ void st16(void* p, u32x4 v) { *reinterpret_cast<u32x4*>(p) = v; }

// bf16 <-> fp32.  Widening is exact; narrowing rounds to nearest, ties to even
// (inputs here are finite).
__device__ __forceinline__ float bf16_to_f32(uint16_t b) { return __uint_as_float(uint32_t(b) << 16); }
__device__ __forceinline__ uint16_t f32_to_bf16(float f) {
  uint32_t u = __float_as_uint(f);
  u += 0x7FFFu + ((u >> 16) & 1u);
  return uint16_t(u >> 16);
}

template <typename T> struct Elem;
template <> struct Elem<float> {
  static __device__ __forceinline__ float to_f32(float v) { return v; }
};
template <> struct Elem<uint16_t> {
  static __device__ __forceinline__ float to_f32(uint16_t v) { return bf16_to_f32(v); }
};

// Lanes e >= 0 (an expert id < 64; -1 = none) of a wave: the rank of this
// lane among the lanes with the same id (lower lanes first), and in `cnt` the
// size of that group.  The lanes whose id equals this lane's are the AND over
// the six bits of the id of the bit's ballot, complemented where this lane's
// bit is 0.  lt_mask = the lanes below this one.
__device__ __forceinline__ int wave_rank(int e, uint64_t lt_mask, int& cnt) {
  const uint64_t valid = __ballot(e >= 0);
  uint32_t lo = (uint32_t)valid, hi = (uint32_t)(valid >> 32);
#pragma unroll
  for (int b = 0; b < 6; ++b) {
    const uint64_t bb = __ballot((e >> b) & 1);
    const uint32_t flip = ((uint32_t)(e >> b) & 1u) - 1u;   // 0 where the bit is set, else ~0
    lo &= (uint32_t)bb ^ flip;
    hi &= (uint32_t)(bb >> 32) ^ flip;
  }
  const uint64_t same = ((uint64_t)hi << 32) | lo;
  cnt = __popcll(same);
  return __popcll(same & lt_mask);
}

// Lanes e >= 0 (an expert id < 64; -1 = none) of a wave: how many lanes hold
// id x, returned in lane x (the same bit-ballot match, against x's bits).
__device__ __forceinline__ int wave_count_of_lane(int e, int lane) {
  const uint64_t valid = __ballot(e >= 0);
  uint32_t lo = (uint32_t)valid, hi = (uint32_t)(valid >> 32);
#pragma unroll
  for (int b = 0; b < 6; ++b) {
    const uint64_t bb = __ballot((e >> b) & 1);
    const uint32_t flip = ((uint32_t)(lane >> b) & 1u) - 1u;
    lo &= (uint32_t)bb ^ flip;
    hi &= (uint32_t)(bb >> 32) ^ flip;
  }
  return __popcll(((uint64_t)hi << 32) | lo);
}

// One 16x16 output tile, K = 32 (bf16) per instruction.  Operand lane layout:
// lane l holds row/column (l % 16) and the 8 consecutive k-slots 8*(l/16)..+7.
// Since the product sums over k, the kernels may map k-slots to any k as long
// as A and B use the same map.
__device__ __forceinline__ f32x4 mfma_bf16(u32x4 a, u32x4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                 __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}
// fp32 variant, K = 4 per instruction: lane l holds row/column (l % 16), k-slot l/16.
__device__ __forceinline__ f32x4 mfma_f32(float a, float b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0);
}
// Output layout of both: lane l holds column (l % 16), rows 4*(l/16) + i, i = 0..3.

typedef float f32x16 __attribute__((ext_vector_type(16)));
// One 32x32 output tile, K = 16 (bf16) per instruction.  Operand lane layout:
// lane l holds row/column (l % 32) and k-slots 8*(l/32)..+7.  Output: lane l,
// register i holds row 8*(i/4) + 4*(l/32) + (i%4), column l % 32.  From a
// single wave per SIMD this shape keeps the matrix pipe ~85% busy, the
// 16x16x32 shape only ~53% (measured on MI355X), so the MFMA-bound kernel uses it.
__device__ __forceinline__ f32x16 mfma32_bf16(u32x4 a, u32x4 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a),
                                                 __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// GELU(z) = z * Phi(z) = (z / 2) * (1 + erf(z / sqrt 2)), with erf from
// Abramowitz & Stegun, Handbook of Mathematical Functions, formula 7.1.26
// (after Hastings): for a >= 0, erfc(a) ~= t P(t) exp(-a^2) with t = 1/(1 + p a)
// and P a fourth-degree polynomial; |error| <= 1.5e-7.  With a = |z| / sqrt 2
// and r = erfc(a) / 2:  GELU(z) = z - z r for z >= 0 and z r for z < 0
// (1 + erf(-a) = erfc(a)), i.e. max(z, 0) - |z| r in both cases (one fused
// multiply-add, no select), so there is no cancellation and GELU's absolute
// error stays below ~1e-7 |z|.  The 1/sqrt 2 is folded into p, the 1/2 into
// P's coefficients, and exp(-a^2) = exp2(-z^2 log2(e) / 2).
__device__ __forceinline__ float gelu_erf(float z) {
  constexpr float kP = 0.3275911f * 0.70710678118654752440f;
  constexpr float c1 = 0.5f * 0.254829592f, c2 = 0.5f * -0.284496736f, c3 = 0.5f * 1.421413741f,
                  c4 = 0.5f * -1.453152027f, c5 = 0.5f * 1.061405429f;
  const float t = __builtin_amdgcn_rcpf(fmaf(kP, fabsf(z), 1.0f));
  float q = fmaf(c5, t, c4);
  q = fmaf(q, t, c3);
  q = fmaf(q, t, c2);
  q = fmaf(q, t, c1);
  q *= t;
  const float e = __builtin_amdgcn_exp2f(z * z * -0.72134752044448170368f);
  return fmaf(-fabsf(z), q * e, fmaxf(z, 0.f));
}

// The same for a result that is rounded to bf16 next: Phi(-|z|) = exp2(q(|z|)) with q of
// degree 7 fitted to log2 Phi(-x) on [0, 7], so one transcendental instead of two.  Relative
// error of the term |z| Phi(-|z|) under 1.3e-5 there, 1/300 of the rounding's; past 7, where
// the term itself is under 1e-11, q falls on to -inf.  Positive z is cut at 1e4 in the term
// (0 from far below), so that +inf stays +inf; -inf and NaN give NaN, as z Phi(z) does.
__device__ __forceinline__ float gelu_for_bf16(float z) {
  const float x = fabsf(__builtin_elementwise_minimum(z, 1e4f));   // keeps NaN, as fminf would not
  float q = fmaf(-1.5882183106441516e-06f, x, 5.615340342046693e-05f);
  q = fmaf(q, x, -0.0008832158055156469f);
  q = fmaf(q, x, 0.008303220383822918f);
  q = fmaf(q, x, -0.053501322865486145f);
  q = fmaf(q, x, -0.4589643180370331f);
  q = fmaf(q, x, -1.1510356664657593f);
  q = fmaf(q, x, -1.0000139474868774f);
  return fmaf(-x, __builtin_amdgcn_exp2f(q), fmaxf(z, 0.f));
}

// Two fp32 values rounded to bf16 (nearest, ties to even) and packed, lo in
// bits 0..15: one v_cvt_pk_bf16_f32 on gfx950.
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2){lo, hi}, bf16x2));
}

// global -> LDS, 16 B per lane to lds_addr + lane * 16, from a uniform base and a 32-bit
// lane offset.  The compiler sees no LDS write: the kernel waits for vmcnt itself
// (wait_vm: at most vm vector-memory operations outstanding).
__device__ __forceinline__ void dma16(const void* base, uint32_t off, uint32_t lds_addr) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1"
               :: "v"(off), "s"(base), "s"(lds_addr) : "memory", "m0");
}
constexpr int wait_vm(int vm) { return (vm & 0xF) | ((vm >> 4) << 14) | (0x7 << 4) | (0xF << 8); }
constexpr int wait_vm_lgkm0(int vm) { return (vm & 0xF) | ((vm >> 4) << 14) | (0x7 << 4); }

// Reductions over the 64 lanes with DPP moves (a few cycles each, where a shuffle goes
// through LDS): pairs, quads, eights and rows of 16 by permutation, then rows 0 -> 1 and
// 2 -> 3, then the lower half into the upper; lane 63 holds the result, returned to all.
template <typename F>
__device__ __forceinline__ uint32_t wave_reduce(uint32_t v, uint32_t unit, F f) {
  v = f(v, (uint32_t)__builtin_amdgcn_update_dpp((int)unit, (int)v, 0xB1, 0xF, 0xF, false));   // quad [1,0,3,2]
  v = f(v, (uint32_t)__builtin_amdgcn_update_dpp((int)unit, (int)v, 0x4E, 0xF, 0xF, false));   // quad [2,3,0,1]
  v = f(v, (uint32_t)__builtin_amdgcn_update_dpp((int)unit, (int)v, 0x141, 0xF, 0xF, false));  // half-row mirror
  v = f(v, (uint32_t)__builtin_amdgcn_update_dpp((int)unit, (int)v, 0x140, 0xF, 0xF, false));  // row mirror
  v = f(v, (uint32_t)__builtin_amdgcn_update_dpp((int)unit, (int)v, 0x142, 0xA, 0xF, false));  // row_bcast15
  v = f(v, (uint32_t)__builtin_amdgcn_update_dpp((int)unit, (int)v, 0x143, 0xC, 0xF, false));  // row_bcast31
  return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}
__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {
  return wave_reduce(v, 0u, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
}
__device__ __forceinline__ float wave_max_f(float v) {
  return __uint_as_float(wave_reduce(__float_as_uint(v), 0xff800000u, [](uint32_t a, uint32_t b) {
    return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
  }));
}
__device__ __forceinline__ float wave_sum_f(float v) {
  return __uint_as_float(wave_reduce(__float_as_uint(v), 0u, [](uint32_t a, uint32_t b) {
    return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
  }));
}

// e^x within ~2 ulp for |x| < 88: 2^(x log2 e) with the rounding error of the product put
// back to first order.  From 88 to 88.72, where it overflows, without that (3e-6 relative);
// below -87.34 it is under fp32's normal range.  Infinities and NaN come out as they should.
__device__ __forceinline__ float exp_f32(float x) {
  constexpr float kL = 1.44269504088896340736f, kLo = 1.92596299112661746887e-8f, kLn2 = 0.69314718055994530942f;
  const float t = x * kL;
  const float e = fmaf(x, kLo, fmaf(x, kL, -t));
  const float r = __builtin_amdgcn_exp2f(t);
  return fabsf(x) < 88.f ? fmaf(r, e * kLn2, r) : r;
}
__device__ __forceinline__ float sigmoid_f32(float x) { return __builtin_amdgcn_rcpf(1.f + exp_f32(-x)); }

// sigmoid(x) and 1 - sigmoid(x), each to fp32: the difference itself would keep few bits of it.
__device__ __forceinline__ void sigmoid_pair(float x, float& s, float& rest) {
  const float t = exp_f32(-fabsf(x)), big = 1.f / (1.f + t), small = t * big;
  s = x < 0.f ? small : big;
  rest = x < 0.f ? big : small;
}

__device__ __forceinline__ int lane_id() { return __lane_id(); }

}  // namespace moe
