// Grouped expert products with MXFP4 weights, many rows per expert: LDS-tiled.
//
// Block tile BM rows of one expert x 256 output columns, 4 waves as 2 x 2, one wave per
// SIMD, each with BM/2 x 128 outputs as 32x32 MFMA tiles in fp32 accumulators.  The MFMA
// takes W rows as its first operand, so a lane holds four consecutive columns of a row.
//   fp4 activations:  steps of 256 k, v_mfma_scale_f32_32x32x64_f8f6f4 with both
//                     operands e2m1 and a scale byte per lane (its 32 values of k);
//   bf16 activations: steps of 64 k, codes widened in registers to bf16 (exact, scale
//                     included) one slice ahead of v_mfma_f32_32x32x16_bf16.  The k of a
//                     slice is free as long as both operands agree: lane half h takes
//                     k = 32 h + 8 s .. + 7 for slice s, so one 16-byte read of a code row
//                     serves the lane's whole step and has one scale.
//
// What bounds the loads is cache lines, not bytes: measured on MI355X, LDS loads from L2
// move about one line per ns and CU, whole or in part (rows of 128 B 127 B/ns, of 64 B
// 65 B/ns, single dwords 4 B/ns).  So rows are read 128 B at a time where LDS allows it,
// and the scales, which the caller has by rows (a line per row for 8 useful bytes), are
// first copied to [k / 256][row][8 bytes], which a tile reads in whole lines.
//
// Persistent blocks, one per CU: the loads run S - 1/2 steps ahead of the products and go
// on into the block's next tile, so its first steps arrive while this tile's results are
// finished and stored.  One barrier per step, before its last part: by then the next step
// has landed, everyone has read the last of this one, and its stage is refilled.
//
// fp4: 32768 rows, K = 4096, N = 14336 1197 to 1278 us by the box, 3.1 PFLOP/s; random codes
// hold the chip at 1.8 GHz (the MFMA alone reaches 6.35 PFLOP/s on them, 8.9 on zeros).  About
// a quarter of the time is the tiles' ends, GELU and 940 MB of stores, which nothing overlaps:
// the accumulators fill the matrix cores' registers, and a tile's end waits for its own stores
// (they and the bias loads of the next 32 columns, or the next step's loads, share a counter).  (Keeping packed results to store them
// during the next tile: 1488 us; 128-row tiles with the end left out altogether: no faster
// than this.)  bf16: 8192 rows, K = 1024, N = 4096 109 us, 0.63 PFLOP/s; K = 4096 1.3.
//
// LDS banks: 16-byte chunks of a row sit at chunk ^ f(row) such that 16 consecutive rows'
// reads of one chunk touch every bank once (128 B rows: (row >> 1) & 7; 32 B rows:
// (row >> 3) & 1).
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "device_common.h"
#include "mx.h"
#include "mx_tiles.h"

namespace moe {

constexpr int kXcd = 8, kBand = 4;
constexpr int kTileN = 256;
constexpr int kCus = 256;           // one block per CU

typedef int i32x8 __attribute__((ext_vector_type(8)));

// First operand codes `w` with scale byte WB of ws, second `a` with byte AB of as.
template <int BYTE>
__device__ __forceinline__ f32x16 mfma_fp4(u32x4 w, int ws, u32x4 a, int as, f32x16 c) {
  const i32x8 x = {(int)w[0], (int)w[1], (int)w[2], (int)w[3], 0, 0, 0, 0};
  const i32x8 y = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(x, y, c, 4, 4, BYTE, ws, BYTE, as);
}

// Tile of block b: XCD b % 8 owns 4 m-tiles of every group of 32 and walks them n-tile by
// n-tile, so the blocks it runs together share their rows in its L2 and all XCDs sweep the
// same columns of W; leftover m-tiles are dealt round-robin.
__device__ __forceinline__ bool tile_of(int total, int ntn, int b, int& mt, int& nt) {
  constexpr int kGroup = kXcd * kBand;
  const int x = b % kXcd, i = b / kXcd;
  const int G = total / kGroup, full = G * kBand * ntn, lm = total - G * kGroup;
  if (i < full) {
    const int g = i / (kBand * ntn), rem = i - g * kBand * ntn;
    nt = rem / kBand;
    mt = g * kGroup + x * kBand + rem % kBand;
    return true;
  }
  const int u = (i - full) * kXcd + x;
  if (u >= lm * ntn) return false;
  nt = u / lm;
  mt = G * kGroup + u % lm;
  return true;
}

static long tile_blocks(long total, long ntn) {
  const long G = total / (kXcd * kBand), lm = total % (kXcd * kBand);
  return kXcd * (G * kBand * ntn + (lm * ntn + kXcd - 1) / kXcd);
}

struct TileArgs {
  const uint8_t* a;        // codes [rows][K/2], or bf16 [rows][K]
  const uint8_t* as;       // scales of the dispatched rows [K/256][rows][8] (FP4)
  const int32_t* src;      // or null
  int k_top, tokens;
  const int32_t* offsets;
  int E, rows, N, K;
  const uint8_t* w;
  const uint8_t* ws;       // scales [E][K/256][N][8]
  const uint16_t* bias;
  void* out;
};

// Scales by rows ([row][K/32]) to groups of 256 k: [K/256 rounded up][row][8], dword h the
// bytes of blocks h, h + 2, h + 4, h + 6 (the ones lane half h of the four slices of 64 k
// needs); blocks past K are 0 (2^-127).  A block turns 64 rows x 16 groups through LDS, so both
// sides go by whole cache lines; the first `w_blocks` take the weights (N rows per expert, a
// multiple of 64), the rest the dispatched rows of the activations.
__global__ __launch_bounds__(256) void mx_scale_groups_kernel(
    const uint8_t* __restrict__ ws, uint8_t* __restrict__ w_out, int w_blocks, int N,
    const uint8_t* __restrict__ as, uint8_t* __restrict__ a_out, int rows,
    const int32_t* __restrict__ src, int k_top, int tokens, int K) {
  __shared__ uint2 turn[16][65];
  const int tid = threadIdx.x, groups = (K + 255) / 256, pitch = K / 32;
  const bool weights = (int)blockIdx.x < w_blocks;
  const int all = weights ? N : rows;                  // rows of the output
  const int per = N / 64, e = weights ? blockIdx.x / per : 0;
  const int r0 = (weights ? blockIdx.x - e * per : blockIdx.x - w_blocks) * 64, g0 = blockIdx.y * 16;
  const uint8_t* in = weights ? ws + (size_t)e * N * pitch : as;
  uint8_t* out = weights ? w_out + (size_t)e * groups * N * 8 : a_out;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = i * 16 + (tid >> 4), g = g0 + (tid & 15);
    if (r0 + r >= all || g >= groups) continue;
    const int from = !weights && src ? (int)min((uint32_t)src[r0 + r] / (uint32_t)k_top, (uint32_t)tokens - 1u) : r0 + r;
    const uint8_t* at = in + (size_t)from * pitch + g * 8;
    const uint32_t lo = *reinterpret_cast<const uint32_t*>(at);
    const uint32_t hi = g * 8 + 4 < pitch ? *reinterpret_cast<const uint32_t*>(at + 4) : 0u;
    turn[tid & 15][r] = make_uint2(__builtin_amdgcn_perm(hi, lo, 0x06040200), __builtin_amdgcn_perm(hi, lo, 0x07050301));
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = tid & 63, g = i * 4 + (tid >> 6);
    if (r0 + r < all && g0 + g < groups)
      *reinterpret_cast<uint2*>(out + ((size_t)(g0 + g) * all + r0 + r) * 8) = turn[g][r];
  }
}

template <bool FP4, bool UP, int BM>
__global__ __launch_bounds__(256, 1) void mx_tile_kernel(TileArgs p) {
  constexpr int S = FP4 ? 2 : 3;
  constexpr int KS = FP4 ? 256 : 64;                             // k per step
  constexpr int kWRow = FP4 ? 128 : 32;                          // bytes of a W row per step
  constexpr int kA = BM * 128, kW = kTileN * kWRow;
  constexpr int kSA = FP4 ? BM * 8 : 0, kSW = kTileN * 8;
  constexpr int kStage = kA + kW + kSA + kSW;
  constexpr int oW = kA, oSA = kA + kW, oSW = oSA + kSA;
  constexpr int kAI = kA / 4096, kWI = kW / 4096;                // 1 KB loads per wave
  constexpr int L = kAI + kWI + 1;
  constexpr int kMT = BM / 64, kNT = 4;                          // 32x32 tiles per wave
  constexpr int kM = kMT * kNT;                                  // MFMAs per slice
  static_assert(S * kStage + sizeof(TileTable) <= 160 * 1024 && kAI >= 1, "LDS plan");
  __shared__ __attribute__((aligned(1024))) uint8_t lds[S * kStage];
  __shared__ TileTable table;

  const int N = p.N, K = p.K, ntn = (N + kTileN - 1) / kTileN;
  const int nk = (K + KS - 1) / KS;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 1, wn = wave & 1, fr = lane & 31, fc = lane >> 5;
  const uint32_t lds0 = (uint32_t)(uintptr_t)lds;
  const uint32_t a_pitch = FP4 ? K / 2 : K * 2, w_pitch = K / 2;

  // ---- the tile being loaded: 32-bit lane offsets from uniform bases that advance ----
  const int total = fill_tiles<BM>(p.offsets, p.E, p.rows, table);
  struct Where {
    int e, r0, r1, n0;
  };
  int b = blockIdx.x;
  auto locate = [&](Where& w) {
    int mt, nt;
    if (!tile_of(total, ntn, b, mt, nt)) return false;
    if (!find_tile<BM>(table, mt, w.e, w.r0, w.r1)) return false;
    w.n0 = nt * kTileN;
    return true;
  };
  // W rows of load i: 4 kPer i + those of load 0, one lane offset; where the tile's second
  // 128 columns are past N its first 128 are read again.
  constexpr int kWLanes = kWRow / 16, kWPer = 64 / kWLanes;
  uint32_t a_off[kAI];
  const int w_row0 = wave * kWPer + lane / kWLanes;
  const uint32_t w_off = (uint32_t)w_row0 * w_pitch +
                         (((lane % kWLanes) ^ (FP4 ? (w_row0 >> 1) & 7 : (w_row0 >> 3) & 1)) << 4);
  uint32_t w_wrap;                                               // bytes to go back
  const uint8_t *w_base, *s_base;                                // s_base: this wave's scales
  size_t s_step;                                                 // bytes per group of 256 k
  auto aim = [&](const Where& w) {
    int g[kAI];
#pragma unroll
    for (int i = 0; i < kAI; ++i) g[i] = min(w.r0 + (i * 4 + wave) * 8 + (lane >> 3), w.r1 - 1);
    if (UP && p.src) {
#pragma unroll
      for (int i = 0; i < kAI; ++i) g[i] = p.src[g[i]];
#pragma unroll
      for (int i = 0; i < kAI; ++i)
        g[i] = (int)min((uint32_t)g[i] / (uint32_t)p.k_top, (uint32_t)p.tokens - 1u);
    }
#pragma unroll
    for (int i = 0; i < kAI; ++i) {
      const int row = (i * 4 + wave) * 8 + (lane >> 3);
      a_off[i] = (uint32_t)g[i] * a_pitch + (((lane & 7) ^ ((row >> 1) & 7)) << 4);
    }
    w_base = p.w + ((size_t)w.e * N + w.n0) * w_pitch;
    w_wrap = N - w.n0 < kTileN ? 128u * w_pitch : 0u;
    // One 1 KB load of scales (128 rows) per wave and step: the first two waves the
    // activations' (FP4; BM = 128: both the same), the others the weights'.
    if (FP4 && wave < 2) {
      s_base = p.as + ((size_t)w.r0 + (wave * 128) % BM) * 8;
      s_step = (size_t)p.rows * 8;
    } else {
      s_base = p.ws + (((size_t)w.e * ((K + 255) / 256)) * N + w.n0 + (wave & 1) * 128) * 8;
      s_step = (size_t)N * 8;
    }
  };
  const uint32_t s_lds = (FP4 && wave < 2) ? oSA + (wave * 1024) % (kSA ? kSA : 1) : oSW + (wave & 1) * 1024;
  // FP4 and K an odd multiple of 128: the last step's chunks past the row's end read the
  // row's first half of that step instead; their scales are 0.
  const uint32_t past_end = (FP4 && ((lane & 7) ^ ((wave * 4 + (lane >> 4)) & 7)) >= 4) ? 64u : 0u;

  Where cur, next;
  if (!locate(cur)) return;
  next = cur;
  bool more = true;                                              // the loads have a tile
  aim(cur);
  int ls = 0;                                                    // its step
  auto load = [&](int i, int stage, uint32_t back) {
    const uint32_t base = lds0 + stage * kStage;
    if (i < kAI) {
      dma16(p.a + (size_t)ls * 128, a_off[i < kAI ? i : 0] - back, base + (i * 4 + wave) * 1024);
    } else if (i < kAI + kWI) {
      const int j = i - kAI;
      const uint32_t row = (uint32_t)(j * 4 * kWPer) * w_pitch - (j * 4 * kWPer >= 128 ? w_wrap : 0u);
      dma16(w_base + row + (size_t)ls * kWRow, w_off - back, base + oW + (j * 4 + wave) * 1024);
    } else {
      dma16(s_base + (FP4 ? ls : ls >> 2) * s_step, (uint32_t)lane * 16, base + s_lds);
    }
  };
  auto back_of = [&]() -> uint32_t { return (FP4 && (K & 128) && ls == nk - 1) ? past_end : 0u; };
  // After a step's loads: on to the next step, or tile; past the last tile the last step
  // is loaded again (those loads land in a free stage and are never read).
  auto advance = [&]() {
    if (++ls < nk) return;
    if (more) {
      b += gridDim.x;
      Where w;
      more = locate(w);
      if (more) {
        next = w;
        aim(w);
        ls = 0;
        return;
      }
    }
    ls = nk - 1;
  };

  f32x16 acc[kNT][kMT];
  // Fragment addresses: rows 32 apart share their swizzle, so a slice has one lane offset.
  const uint32_t f_swz = (fr >> 1) & 7;
  const uint32_t a_lane = (uint32_t)(wm * (BM / 2) + fr) * 128, w_lane = (uint32_t)(wn * 128 + fr) * kWRow;
  auto read_a = [&](int stage, int m, int chunk) {
    return ld16(lds + (stage * kStage + a_lane + ((chunk ^ f_swz) << 4)) + m * 4096);
  };
  auto read_w = [&](int stage, int j, int chunk) {
    const uint32_t c = (chunk ^ (FP4 ? f_swz : (uint32_t)(fr >> 3) & 1u)) << 4;
    return ld16(lds + (stage * kStage + w_lane + c) + oW + j * 32 * kWRow);
  };
  auto read_sa = [&](int stage, int m) {
    return *reinterpret_cast<const int*>(lds + (stage * kStage + (wm * (BM / 2) + fr) * 8 + fc * 4) + oSA + m * 256);
  };
  auto read_sw = [&](int stage, int j) {
    return *reinterpret_cast<const int*>(lds + (stage * kStage + (wn * 128 + fr) * 8 + fc * 4) + oSW + j * 256);
  };

  // Epilogue of the tile at `w`: bias, GELU, stores straight from the accumulators, which
  // neither wait for LDS nor need any.  A lane has columns 8g + 4fc .. + 3 of its row; fp32
  // stores them as they are, bf16 first swaps between the lane halves, so that one has all 8
  // columns of g and the other those of g + 1 (32 bytes of each row per store either way).
  auto finish = [&](const Where& w) {
#pragma unroll
    for (int j = 0; j < kNT; ++j) {
      const int col0 = w.n0 + wn * 128 + j * 32;
      uint2 braw[4];
#pragma unroll
      for (int g = 0; g < 4; ++g)
        braw[g] = (p.bias && col0 < N)
                      ? *reinterpret_cast<const uint2*>(p.bias + (size_t)w.e * N + col0 + 8 * g + 4 * fc)
                      : make_uint2(0u, 0u);
#pragma unroll
      for (int m = 0; m < kMT; ++m) {
        const int r = w.r0 + wm * (BM / 2) + m * 32 + fr;
        const bool in = r < w.r1 && col0 < N;
        // Out of the matrix cores' registers one tile at a time: all at once would spill.
        asm volatile("" : "+a"(acc[j][m]));
        f32x4 v[4];
#pragma unroll
        for (int g = 0; g < 4; ++g) {
#pragma unroll
          for (int q = 0; q < 4; ++q) v[g][q] = acc[j][m][4 * g + q];
          v[g][0] += __uint_as_float(braw[g].x << 16);
          v[g][1] += __uint_as_float(braw[g].x & 0xffff0000u);
          v[g][2] += __uint_as_float(braw[g].y << 16);
          v[g][3] += __uint_as_float(braw[g].y & 0xffff0000u);
        }
        if constexpr (UP) {
          uint16_t* o = static_cast<uint16_t*>(p.out) + (size_t)r * N + col0 + 8 * fc;
#pragma unroll
          for (int g = 0; g < 4; g += 2) {
            uint32_t h[2][2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              h[i][0] = pack_bf16x2(gelu_for_bf16(v[g + i][0]), gelu_for_bf16(v[g + i][1]));
              h[i][1] = pack_bf16x2(gelu_for_bf16(v[g + i][2]), gelu_for_bf16(v[g + i][3]));
            }
            const auto s0 = __builtin_amdgcn_permlane32_swap(h[0][0], h[1][0], false, false);
            const auto s1 = __builtin_amdgcn_permlane32_swap(h[0][1], h[1][1], false, false);
            if (in) st16(o + 8 * g, u32x4{s0[0], s1[0], s0[1], s1[1]});
          }
        } else {
          float* o = static_cast<float*>(p.out) + (size_t)r * N + col0 + 4 * fc;
#pragma unroll
          for (int g = 0; g < 4; ++g)
            if (in) *reinterpret_cast<f32x4*>(o + 8 * g) = v[g];
        }
      }
    }
  };

  // ---- prologue: every stage but the last in full, of the last its first LA loads ----
  constexpr int LA = FP4 ? (L + 1) / 2 : L;   // FP4: the rest goes with the next step's start
#pragma unroll
  for (int s = 0; s < S; ++s) {
    const uint32_t back = back_of();
#pragma unroll
    for (int i = 0; i < L; ++i)
      if (s < S - 1 || i < LA) load(i, s, back);
    if (s < S - 1 || LA == L) advance();
  }
  __builtin_amdgcn_s_waitcnt(wait_vm((S - 2) * L + LA));
  __syncthreads();

  int st = 0;                                          // stage of the step being multiplied
  if constexpr (FP4) {
    u32x4 xa[kMT], xw[kNT], ya[kMT], yw[kNT];
    int sa[kMT], sw[kNT];
#pragma unroll
    for (int m = 0; m < kMT; ++m) xa[m] = read_a(0, m, fc), sa[m] = read_sa(0, m);
#pragma unroll
    for (int j = 0; j < kNT; ++j) xw[j] = read_w(0, j, fc), sw[j] = read_sw(0, j);
    for (;;) {
#pragma unroll
      for (int j = 0; j < kNT; ++j)
#pragma unroll
        for (int m = 0; m < kMT; ++m)
#pragma unroll
          for (int q = 0; q < 16; ++q) acc[j][m][q] = 0.f;
      const Where done = cur;
      bool go_on = false;
      for (int t = 0; t < nk; ++t) {
        // Slice 0: the rest of the pending step's loads (into the other stage).
        {
          const uint32_t back = back_of();
#pragma unroll
          for (int q = 0; q < kM; ++q) {
            const int j = q / kMT, m = q % kMT;
            acc[j][m] = mfma_fp4<0>(xw[j], sw[j], xa[m], sa[m], acc[j][m]);
            if (q < kMT) ya[q] = read_a(st, q, 2 + fc);
            if (q < kNT) yw[q] = read_w(st, q, 2 + fc);
#pragma unroll
            for (int i = LA + q * (L - LA) / kM; i < LA + (q + 1) * (L - LA) / kM; ++i) load(i, st ^ 1, back);
            __builtin_amdgcn_sched_barrier(0);
          }
        }
#pragma unroll
        for (int q = 0; q < kM; ++q) {
          const int j = q / kMT, m = q % kMT;
          acc[j][m] = mfma_fp4<1>(yw[j], sw[j], ya[m], sa[m], acc[j][m]);
          if (q < kMT) xa[q] = read_a(st, q, 4 + fc);
          if (q < kNT) xw[q] = read_w(st, q, 4 + fc);
          __builtin_amdgcn_sched_barrier(0);
        }
        advance();
        if (t == nk - 1) go_on = more;
#pragma unroll
        for (int q = 0; q < kM; ++q) {
          const int j = q / kMT, m = q % kMT;
          acc[j][m] = mfma_fp4<2>(xw[j], sw[j], xa[m], sa[m], acc[j][m]);
          if (q < kMT) ya[q] = read_a(st, q, 6 + fc);
          if (q < kNT) yw[q] = read_w(st, q, 6 + fc);
          __builtin_amdgcn_sched_barrier(0);
        }
        __builtin_amdgcn_s_waitcnt(wait_vm_lgkm0(0));
        __syncthreads();
        // Slice 3: the next step's first fragments and scales, loads into this stage.
        int na[kMT], nw[kNT];
        const uint32_t back = back_of();
#pragma unroll
        for (int q = 0; q < kM; ++q) {
          const int j = q / kMT, m = q % kMT;
          acc[j][m] = mfma_fp4<3>(yw[j], sw[j], ya[m], sa[m], acc[j][m]);
          if (q < kMT) xa[q] = read_a(st ^ 1, q, fc), na[q] = read_sa(st ^ 1, q);
          if (q < kNT) xw[q] = read_w(st ^ 1, q, fc), nw[q] = read_sw(st ^ 1, q);
#pragma unroll
          for (int i = q * LA / kM; i < (q + 1) * LA / kM; ++i) load(i, st, back);
          __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int m = 0; m < kMT; ++m) sa[m] = na[m];
#pragma unroll
        for (int j = 0; j < kNT; ++j) sw[j] = nw[j];
        st ^= 1;
      }
      finish(done);
      if (!go_on) break;
      cur = next;
    }
  } else {
    u32x4 xa[2][kMT], ya[2][kMT], raw[kNT], wf[2][kNT];
    float sc[kNT];
    auto widen = [&](const u32x4 (&r)[kNT], const float (&s)[kNT], u32x4 (&to)[kNT], int slice, int i) {
      const int j = i / 4, q = i % 4;
      uint32_t v;
      const uint32_t c = r[j][slice];
      if (q == 0) v = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s[j], 0));
      else if (q == 1) v = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s[j], 1));
      else if (q == 2) v = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s[j], 2));
      else v = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s[j], 3));
      to[j][q] = v;
    };
    // The scale of step t: byte t % 4 of its group's dword.
    auto scale_of = [&](int v, int t) { return __uint_as_float((((uint32_t)v >> (8 * (t & 3))) & 0xffu) << 23); };
#pragma unroll
    for (int m = 0; m < kMT; ++m) xa[0][m] = read_a(0, m, 4 * fc), xa[1][m] = read_a(0, m, 4 * fc + 1);
#pragma unroll
    for (int j = 0; j < kNT; ++j) raw[j] = read_w(0, j, fc), sc[j] = scale_of(read_sw(0, j), 0);
#pragma unroll
    for (int i = 0; i < 4 * kNT; ++i) widen(raw, sc, wf[0], 0, i);
    constexpr int kCv = 4 * kNT;                       // conversions per slice
    for (;;) {
#pragma unroll
      for (int j = 0; j < kNT; ++j)
#pragma unroll
        for (int m = 0; m < kMT; ++m)
#pragma unroll
          for (int q = 0; q < 16; ++q) acc[j][m][q] = 0.f;
      const Where done = cur;
      bool go_on = false;
      for (int t = 0; t < nk; ++t) {
        const int st1 = st == S - 1 ? 0 : st + 1;
        // Slices 0 and 1; reads of slices 2 and 3; conversions of slices 1 and 2.
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
          for (int q = 0; q < kM; ++q) {
            const int j = q / kMT, m = q % kMT;
            acc[j][m] = mfma32_bf16(wf[s][j], xa[s][m], acc[j][m]);
#pragma unroll
            for (int i = q * kCv / kM; i < (q + 1) * kCv / kM; ++i) widen(raw, sc, wf[s ^ 1], s + 1, i);
            if (s == 0 && q < kMT) ya[0][q] = read_a(st, q, 4 * fc + 2), ya[1][q] = read_a(st, q, 4 * fc + 3);
            __builtin_amdgcn_sched_barrier(0);
          }
        __builtin_amdgcn_s_waitcnt(wait_vm_lgkm0((S - 2) * L));
        __syncthreads();
        // Slices 2 and 3; the next step's codes, scales and first fragments; loads.
        u32x4 nraw[kNT];
        float nsc[kNT];
        const int tn = t + 1 < nk ? t + 1 : 0;
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
          for (int q = 0; q < kM; ++q) {
            const int j = q / kMT, m = q % kMT;
            acc[j][m] = mfma32_bf16(wf[s][j], ya[s][m], acc[j][m]);
#pragma unroll
            for (int i = q * kCv / kM; i < (q + 1) * kCv / kM; ++i) {
              if (s == 0) widen(raw, sc, wf[1], 3, i);
              else widen(nraw, nsc, wf[0], 0, i);
            }
            if (s == 0 && q < kNT) nraw[q] = read_w(st1, q, fc), nsc[q] = scale_of(read_sw(st1, q), tn);
            if (s == 0 && q < kMT) xa[0][q] = read_a(st1, q, 4 * fc), xa[1][q] = read_a(st1, q, 4 * fc + 1);
            const int at = s * kM + q;
#pragma unroll
            for (int i = at * L / (2 * kM); i < (at + 1) * L / (2 * kM); ++i) load(i, st, 0u);
            __builtin_amdgcn_sched_barrier(0);
          }
#pragma unroll
        for (int j = 0; j < kNT; ++j) raw[j] = nraw[j], sc[j] = nsc[j];
        st = st1;
        advance();
        if (t == nk - 1) go_on = more;
      }
      finish(done);
      if (!go_on) break;
      cur = next;
    }
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");     // no load outlives its LDS
}

template <bool FP4, bool UP, int BM>
static void launch_tile(const TileArgs& p, hipStream_t s) {
  const long most = p.rows / BM + std::min(p.E, p.rows);           // bound on the m-tiles
  const long blocks = tile_blocks(most, (p.N + kTileN - 1) / kTileN);
  mx_tile_kernel<FP4, UP, BM><<<(unsigned)std::min(blocks, (long)kCus), 256, 0, s>>>(p);
}

template <bool FP4, bool UP>
static void launch_tile_rows(const TileArgs& p, int bm, hipStream_t s) {
  if (bm == 256) launch_tile<FP4, UP, 256>(p, s);
  else launch_tile<FP4, UP, 128>(p, s);
}

// Rows per tile, 256 or 128: the estimated rounds of the CUs times a round's time, a part in
// proportion to the height and a fixed one (a tile of 128 rows takes 0.63 of the time of one
// of 256).  The experts' loads differ, so their tiles are counted at 10% less and at 10% more
// than the average.  Measured against both heights at E = 8, 64, 128, 48 to 1024 rows per
// expert, N = 768 to 14336: within 3% of the better one in all 82 cases.  E = 8, K = 4096,
// N = 14336, bf16: 96 rows 139 us of 128 against 208 of 256, 192 rows 250 against 218.
static int tile_height(long rows, int E, int N) {
  const long ntn = (N + kTileN - 1) / kTileN;
  auto time = [&](int bm) {
    const double per = (double)rows / E, off = E > 1 ? 0.1 : 0.0;
    const double tiles = 0.5 * (std::ceil(per * (1 - off) / bm) + std::ceil(per * (1 + off) / bm)) * E * ntn;
    return std::ceil(tiles / kCus) * (bm + 96);
  };
  return time(128) < time(256) ? 128 : 256;
}

// Activation codes and scales (FP4), then the regrouped scales, each padded by one tile's
// worth of rows that the last tile may read past the end.
struct TileSpace {
  size_t scales, a_groups, w_groups, total;
};
static TileSpace tile_space(long rows, int E, int N, int K, bool fp4) {
  auto up256 = [](size_t v) { return (v + 255) & ~size_t(255); };
  const size_t groups = (K + 255) / 256, pad = 256 * 8;
  TileSpace t{};
  t.scales = fp4 ? up256((size_t)rows * K / 2) : 0;
  t.a_groups = t.scales + (fp4 ? up256((size_t)rows * K / 32) : 0);
  t.w_groups = t.a_groups + (fp4 ? up256(groups * rows * 8 + pad) : 0);
  t.total = t.w_groups + up256((size_t)E * groups * N * 8 + pad);
  return t;
}

size_t mx_tile_bytes(long rows, int E, int N, int K, bool fp4) {
  return tile_space(rows, E, N, K, fp4).total;
}

hipError_t launch_mx_tile(const MxFfnArgs& a, hipStream_t s) {
  TileArgs p{};
  p.src = a.up ? a.src : nullptr;
  p.k_top = a.k;
  p.tokens = a.T;
  p.offsets = a.offsets;
  p.E = a.E;
  p.rows = a.T * a.k;
  p.N = a.N;
  p.K = a.K;
  p.w = a.w;
  p.bias = static_cast<const uint16_t*>(a.bias);
  p.out = a.out;
  const TileSpace t = tile_space(p.rows, a.E, a.N, a.K, a.fp4);
  uint8_t* scales = a.act + t.scales;
  uint8_t* a_groups = a.act + t.a_groups;
  uint8_t* w_groups = a.act + t.w_groups;
  p.a = static_cast<const uint8_t*>(a.a);
  if (a.fp4) {
    if (hipError_t e = launch_mx_quantize(a.a, true, a.a_rows, a.K, a.K, a.act, scales, s)) return e;
    p.a = a.act;
    p.as = a_groups;
  }
  p.ws = w_groups;
  const int groups = (a.K + 255) / 256;
  const int w_blocks = a.E * (a.N / 64), a_blocks = a.fp4 ? (p.rows + 63) / 64 : 0;
  mx_scale_groups_kernel<<<dim3(w_blocks + a_blocks, (groups + 15) / 16), 256, 0, s>>>(
      a.ws, w_groups, w_blocks, a.N, scales, a_groups, p.rows, p.src, a.k, a.T, a.K);
  const int bm = tile_height(p.rows, a.E, a.N);
  if (a.fp4)
    a.up ? launch_tile_rows<true, true>(p, bm, s) : launch_tile_rows<true, false>(p, bm, s);
  else
    a.up ? launch_tile_rows<false, true>(p, bm, s) : launch_tile_rows<false, false>(p, bm, s);
  return hipGetLastError();
}

}  // namespace moe
