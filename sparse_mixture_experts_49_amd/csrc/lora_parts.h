// What the kernels of parts share (lora.hip, lora_tile.hip): W x and A x as columns of one product,
// cut along k.
#pragma once

#include "device_common.h"
#include "lora.h"

namespace moe {

// GELU for an fp32 result: +inf stays +inf, as it does for bf16.
__device__ __forceinline__ float gelu_f32(float z) { return z > 1e4f ? z : gelu_erf(z); }

// A block's part: BM tokens, BN columns of W or of the adapters that the tokens have (16 ranks of one
// after the other's), steps [k0, k1) of 64 k.
struct LoraUnit {
  int t0, n0, split, k0, k1;
  bool of_a;
  int g0;                              // of A: its first group of 16 ranks
};

// Block b: the row tiles of one (column tile, part of k) follow one another on one XCD.
template <int BM, int BN>
__device__ __forceinline__ bool lora_unit(const LoraPartArgs& p, LoraUnit& u) {
  const int mts = (p.a.sh.T + BM - 1) / BM, ntn = (p.a.sh.n + BN - 1) / BN, cols = ntn + p.a_tiles;
  const int q = blockIdx.x / 8, cs = q / mts * 8 + blockIdx.x % 8;
  if (cs >= cols * p.splits) return false;
  const int col = cs % cols, nk = p.a.sh.d / 64;
  u.split = cs / cols;
  u.t0 = q % mts * BM;
  u.n0 = col * BN;
  u.of_a = col >= ntn;
  u.g0 = (col - ntn) * (BN / 16);
  u.k0 = (int)((long)u.split * nk / p.splits);
  u.k1 = (int)((long)(u.split + 1) * nk / p.splits);
  return true;
}

// The different adapters among the tokens [t0, t0 + BM), in order of appearance, into list; how
// many.  Every wave does the same.
template <int BM>
__device__ __forceinline__ int lora_list(const LoraArgs& a, int t0, int* list) {
  constexpr int kParts = (BM + 63) / 64;
  const int lane = threadIdx.x & 63;
  int own[kParts];
  uint64_t left[kParts];
#pragma unroll
  for (int i = 0; i < kParts; ++i) {
    const int r = i * 64 + lane;
    own[i] = r < BM && t0 + r < a.sh.T ? a.adapter[t0 + r] : -1;
    left[i] = __ballot((uint32_t)own[i] < (uint32_t)a.sh.N);
  }
  int count = 0;
#pragma unroll
  for (int i = 0; i < kParts; ++i)
    for (; left[i]; ++count) {
      const int one = __builtin_amdgcn_readlane(own[i], __ffsll((unsigned long long)left[i]) - 1);
#pragma unroll
      for (int j = 0; j < kParts; ++j) left[j] &= ~__ballot(own[j] == one);
      list[count] = one;
    }
  return count;
}

}  // namespace moe
