// MXFP4 quantisation on gfx950: blocks of 32 values, one e8m0 scale, e2m1 codes.
//
// scale = 2^(floor(log2 max|x|) - 2): the largest value lands in [4, 8) and 6 is the
// largest code, so what rounds past 6 saturates.  The exponent is read from the bits
// of the maximum, the division by a power of two and the rounding (nearest, ties to
// even) are the conversion instruction's and exact otherwise.
//
// One pass over memory: each lane holds 8 neighbouring values, four lanes make a
// block and exchange their maximum; 16-byte loads, 4-byte code stores.  Bound by memory:
// 57344 x 4096 bf16 values 124 us there (4.8 TB/s read and written, what a copy reaches), 104 us
// back.
#include "device_common.h"
#include "mx.h"

namespace moe {

// Scale byte of a block from the largest magnitude bits (bits of |x| as fp32, so the
// integer maximum is the maximum and NaN and infinity sort last).
__device__ __forceinline__ uint32_t block_scale(uint32_t mag) {
  if (mag >= 0x7f800000u) return 255u;              // NaN or infinity among them
  int e = (int)(mag >> 23);                         // biased floor(log2) of a normal
  return (uint32_t)max(e - 2, 0);                   // subnormals: below 2^-126, clamped too
}

__device__ __forceinline__ uint32_t max4(uint32_t v) {
  v = max(v, (uint32_t)__shfl_xor((int)v, 1));
  return max(v, (uint32_t)__shfl_xor((int)v, 2));
}

// Eight values (two per word, packed conversions) to eight codes.
__device__ __forceinline__ uint32_t codes8(const float (&v)[8], float scale) {
  uint32_t c = 0;
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[0], v[1], scale, 0);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[2], v[3], scale, 1);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[4], v[5], scale, 2);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[6], v[7], scale, 3);
  return c;
}

template <bool BF16>
__device__ __forceinline__ void load8(const void* x, size_t i, float (&v)[8], uint32_t& mag) {
  mag = 0;
  if constexpr (BF16) {
    const u32x4 r = ld16(static_cast<const uint16_t*>(x) + i);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] = __uint_as_float(r[j] << 16);
      v[2 * j + 1] = __uint_as_float(r[j] & 0xffff0000u);
    }
  } else {
    const u32x4 a = ld16(static_cast<const float*>(x) + i), b = ld16(static_cast<const float*>(x) + i + 4);
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = __uint_as_float(a[j]), v[4 + j] = __uint_as_float(b[j]);
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) mag = max(mag, __float_as_uint(v[j]) & 0x7fffffffu);
}

// Thread -> (row, group of 8 columns); cols is a multiple of 32, so the four lanes of a
// block run together.
template <bool BF16>
__global__ __launch_bounds__(256) void mx_quantize_kernel(const void* __restrict__ x, int64_t n8,
                                                          int cols8, int64_t stride,
                                                          uint8_t* __restrict__ codes,
                                                          uint8_t* __restrict__ scales) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= n8) return;
  const int64_t row = i / cols8;
  const int c = (int)(i - row * cols8);
  float v[8];
  uint32_t mag;
  load8<BF16>(x, (size_t)row * stride + c * 8, v, mag);
  const uint32_t sb = block_scale(max4(mag));
  reinterpret_cast<uint32_t*>(codes)[i] = sb == 255u ? 0u : codes8(v, __uint_as_float(sb << 23));
  if ((i & 3) == 0) scales[i >> 2] = (uint8_t)sb;
}

template <bool BF16>
__device__ __forceinline__ void store8(void* out, size_t i, uint32_t c, float scale) {
  // Widened to bf16 (exact) by the conversion instruction, two values at a time.
  u32x4 h;
  h[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 0));
  h[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 1));
  h[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 2));
  h[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 3));
  if constexpr (BF16) {
    st16(static_cast<uint16_t*>(out) + i, h);
  } else {
    u32x4 a, b;
    a[0] = h[0] << 16, a[1] = h[0] & 0xffff0000u, a[2] = h[1] << 16, a[3] = h[1] & 0xffff0000u;
    b[0] = h[2] << 16, b[1] = h[2] & 0xffff0000u, b[2] = h[3] << 16, b[3] = h[3] & 0xffff0000u;
    st16(static_cast<float*>(out) + i, a);
    st16(static_cast<float*>(out) + i + 4, b);
  }
}

template <bool BF16>
__global__ __launch_bounds__(256) void mx_dequantize_kernel(const uint8_t* __restrict__ codes,
                                                            const uint8_t* __restrict__ scales,
                                                            int64_t n8, int cols8, int64_t stride,
                                                            void* __restrict__ out) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= n8) return;
  const int64_t row = i / cols8;
  const int c = (int)(i - row * cols8);
  const float scale = __uint_as_float((uint32_t)scales[i >> 2] << 23);
  store8<BF16>(out, (size_t)row * stride + c * 8, reinterpret_cast<const uint32_t*>(codes)[i], scale);
}

__global__ __launch_bounds__(256) void mx_requantize_kernel(const void* __restrict__ x, int64_t n8,
                                                            void* __restrict__ out) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= n8) return;
  float v[8];
  uint32_t mag;
  load8<true>(x, (size_t)i * 8, v, mag);
  const float scale = __uint_as_float(block_scale(max4(mag)) << 23);
  store8<true>(out, (size_t)i * 8, codes8(v, scale), scale);
}

static unsigned blocks_of(int64_t n) { return (unsigned)((n + 255) / 256); }

hipError_t launch_mx_quantize(const void* x, bool bf16, int64_t rows, int64_t cols, int64_t stride,
                              uint8_t* codes, uint8_t* scales, hipStream_t s) {
  const int64_t n8 = rows * cols / 8;
  if (n8 == 0) return hipSuccess;
  if (bf16)
    mx_quantize_kernel<true><<<blocks_of(n8), 256, 0, s>>>(x, n8, (int)(cols / 8), stride, codes, scales);
  else
    mx_quantize_kernel<false><<<blocks_of(n8), 256, 0, s>>>(x, n8, (int)(cols / 8), stride, codes, scales);
  return hipGetLastError();
}

hipError_t launch_mx_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows,
                                int64_t cols, bool bf16, void* out, int64_t stride, hipStream_t s) {
  const int64_t n8 = rows * cols / 8;
  if (n8 == 0) return hipSuccess;
  if (bf16)
    mx_dequantize_kernel<true><<<blocks_of(n8), 256, 0, s>>>(codes, scales, n8, (int)(cols / 8), stride, out);
  else
    mx_dequantize_kernel<false><<<blocks_of(n8), 256, 0, s>>>(codes, scales, n8, (int)(cols / 8), stride, out);
  return hipGetLastError();
}

hipError_t launch_mx_requantize(const void* x, int64_t rows, int64_t cols, void* out, hipStream_t s) {
  const int64_t n8 = rows * cols / 8;
  mx_requantize_kernel<<<blocks_of(n8), 256, 0, s>>>(x, n8, out);
  return hipGetLastError();
}

}  // namespace moe
