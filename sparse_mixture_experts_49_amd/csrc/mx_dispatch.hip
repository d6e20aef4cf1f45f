// The dispatch layout for up to 256 experts: a stable counting sort of the assignment
// ids by expert, as permute.hip does for 64 (same outputs), without the row gather.
#include "device_common.h"
#include "mx.h"

namespace moe {

constexpr int kMxChunk = 1024;      // assignments per block, 256 per wave

int mx_dispatch_blocks(int assignments) { return (assignments + kMxChunk - 1) / kMxChunk; }

// Rank of this lane among the lanes with its id e in [0, 256) (-1: none), and the size
// of that group: one ballot per bit of the id.
__device__ __forceinline__ int wave_rank8(int e, uint64_t lt_mask, int& cnt) {
  uint64_t same = __ballot(e >= 0);
#pragma unroll
  for (int b = 0; b < 8; ++b) {
    const uint64_t bb = __ballot((e >> b) & 1);
    same &= ((e >> b) & 1) ? bb : ~bb;
  }
  cnt = __popcll(same);
  return __popcll(same & lt_mask);
}

// A wave ranks its 256 assignments in four batches of 64 lanes; wcount[wave] runs the
// counts (this wave's own row, in its program order).
__device__ __forceinline__ void rank_chunk(const int32_t* __restrict__ idx, int A, int E, int base,
                                           int (&ex)[4], int (&rk)[4], int* wrow) {
  const int lane = threadIdx.x & 63;
  const uint64_t lt_mask = lane == 0 ? 0ull : (~0ull >> (64 - lane));
  for (int i = lane; i < kMxMaxExperts; i += 64) wrow[i] = 0;
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    const int a = base + b * 64 + lane;
    const int e = a < A ? idx[a] : -1;
    ex[b] = (e >= 0 && e < E) ? e : -1;
  }
  __builtin_amdgcn_wave_barrier();
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    int cnt;
    const int e = ex[b], within = wave_rank8(e, lt_mask, cnt);
    const int before = e >= 0 ? wrow[e] : 0;
    rk[b] = before + within;
    __builtin_amdgcn_wave_barrier();
    if (e >= 0 && within == 0) wrow[e] = before + cnt;
    __builtin_amdgcn_wave_barrier();
  }
}

// Exclusive prefix of v over the block's 256 threads.
__device__ __forceinline__ int prefix256(int v, int* s, int& total) {
  const int t = threadIdx.x;
  s[t] = v;
  for (int o = 1; o < 256; o <<= 1) {
    __syncthreads();
    const int u = t >= o ? s[t - o] : 0;
    __syncthreads();
    s[t] += u;
  }
  __syncthreads();
  total = s[255];
  const int before = t ? s[t - 1] : 0;
  __syncthreads();
  return before;
}

// SINGLE: one block holds every assignment and does all of it.
template <bool SINGLE>
__global__ __launch_bounds__(256) void mx_rank_kernel(MxDispatchArgs a) {
  __shared__ int wcount[4][kMxMaxExperts];
  __shared__ int first[kMxMaxExperts];              // row of the block's first of expert e
  __shared__ int scan[kMxMaxExperts];
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  const int base = blockIdx.x * kMxChunk + wave * 256;
  int ex[4], rk[4];
  rank_chunk(a.topk_idx, a.A, a.E, base, ex, rk, wcount[wave]);
  __syncthreads();
  if constexpr (SINGLE) {
    const int n = wcount[0][t] + wcount[1][t] + wcount[2][t] + wcount[3][t];
    int total;
    const int off = prefix256(n, scan, total);
    first[t] = off;
    if (t < a.E) a.counts[t] = n, a.offsets[t] = off;
    if (t == 0) a.offsets[a.E] = total;
  } else {
    if (t < a.E) first[t] = a.offsets[t] + a.blk_base[(size_t)blockIdx.x * a.E + t];
  }
  __syncthreads();
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    const int i = base + b * 64 + lane, e = ex[b];
    if (i >= a.A) continue;
    if (e < 0) {
      a.dest[i] = -1;
      continue;
    }
    int row = first[e] + rk[b];
    for (int w = 0; w < wave; ++w) row += wcount[w][e];
    a.dest[i] = row;
    a.src[row] = i;
  }
}

__global__ __launch_bounds__(256) void mx_hist_kernel(MxDispatchArgs a) {
  __shared__ int h[kMxMaxExperts];
  h[threadIdx.x] = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < kMxChunk; i += 256) {
    const int at = blockIdx.x * kMxChunk + i;
    const int e = at < a.A ? a.topk_idx[at] : -1;
    if (e >= 0 && e < a.E) atomicAdd(&h[e], 1);     // counts: order-independent
  }
  __syncthreads();
  if ((int)threadIdx.x < a.E) a.blk_hist[(size_t)blockIdx.x * a.E + threadIdx.x] = h[threadIdx.x];
}

// One thread per expert walks the blocks.
__global__ __launch_bounds__(256) void mx_scan_kernel(MxDispatchArgs a, int blocks) {
  __shared__ int scan[kMxMaxExperts];
  const int t = threadIdx.x;
  int run = 0;
  if (t < a.E)
    for (int b = 0; b < blocks; ++b) {
      const size_t i = (size_t)b * a.E + t;
      a.blk_base[i] = run;
      run += a.blk_hist[i];
    }
  int total;
  const int off = prefix256(run, scan, total);
  if (t < a.E) a.counts[t] = run, a.offsets[t] = off;
  if (t == 0) a.offsets[a.E] = total;
}

hipError_t launch_mx_dispatch(const MxDispatchArgs& a, hipStream_t s) {
  const int nb = mx_dispatch_blocks(a.A);
  if (nb == 1) {
    mx_rank_kernel<true><<<1, 256, 0, s>>>(a);
  } else {
    mx_hist_kernel<<<nb, 256, 0, s>>>(a);
    mx_scan_kernel<<<1, 256, 0, s>>>(a, nb);
    mx_rank_kernel<false><<<nb, 256, 0, s>>>(a);
  }
  return hipGetLastError();
}

}  // namespace moe
