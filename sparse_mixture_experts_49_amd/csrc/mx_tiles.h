// The experts' row segments as row tiles, shared by the MXFP4 products (mx_tile.hip,
// mx_ffn.hip).
#pragma once

#include "device_common.h"

namespace moe {

// The experts' rows cut into m-tiles of BM laid end to end, as a table in LDS: lane l
// holds experts 4l .. 4l+3, entry [i][l] = {first row, end, first m-tile} of 4l + i.
struct TileTable {
  int lo[4][64], hi[4][64], first[4][64];
};

// Every wave writes the same table (no barrier needed); returns the number of m-tiles.
template <int BM>
__device__ __forceinline__ int fill_tiles(const int32_t* __restrict__ offsets, int E, int rows,
                                          TileTable& t) {
  const int lane = __lane_id();
  int first[4], sum = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int e = lane * 4 + i;
    const int lo = e < E ? min(max(offsets[e], 0), rows) : 0;
    const int hi = e < E ? min(max(offsets[e + 1], lo), rows) : 0;
    t.lo[i][lane] = lo;
    t.hi[i][lane] = hi;
    first[i] = sum;
    sum += (hi - lo + BM - 1) / BM;
  }
  int incl = sum;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int v = __shfl_up(incl, o);
    if (lane >= o) incl += v;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) t.first[i][lane] = first[i] + incl - sum;
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  return __builtin_amdgcn_readfirstlane(__shfl(incl, 63));
}

template <int BM>
__device__ __forceinline__ bool find_tile(const TileTable& t, int mt, int& e, int& r0, int& r1) {
  const int lane = __lane_id();
  bool found = false;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int lo = t.lo[i][lane], hi = t.hi[i][lane], first = t.first[i][lane];
    const int n = (hi - lo + BM - 1) / BM;
    const uint64_t own = __ballot(mt >= first && mt < first + n);
    if (own) {
      const int l = __builtin_amdgcn_readfirstlane(__ffsll((unsigned long long)own) - 1);
      e = l * 4 + i;
      r0 = __builtin_amdgcn_readlane(lo + (mt - first) * BM, l);
      r1 = min(__builtin_amdgcn_readlane(hi, l), r0 + BM);
      found = true;
    }
  }
  return found;
}

}  // namespace moe
