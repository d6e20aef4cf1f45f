// Grouped expert products with MXFP4 weights, many rows per expert: LDS-tiled.
//
// Block tile BM rows of one expert x 256 output columns, 4 waves as 2 x 2, one wave per
// SIMD, each with BM/2 x 128 outputs as 32x32 MFMA tiles in fp32 accumulators.  The MFMA
// takes W rows as its first operand, so a lane holds four consecutive columns of a row.
//   FP4 activations:  steps of 128 k, v_mfma_scale_f32_32x32x64_f8f6f4 with both
//                     operands e2m1 and a scale byte per lane (its 32 values of k);
//   bf16 activations: steps of 64 k, codes widened in registers to bf16 (exact, scale
//                     included) one slice ahead of v_mfma_f32_32x32x16_bf16.  The k of a
//                     slice is free as long as both operands agree: lane half h takes
//                     k = 32 h + 8 s .. + 7 for slice s, so one 16-byte read of a code row
//                     serves the lane's whole step and has one scale.
// Operands go from memory straight into a ring of S LDS stages, scales among them
// (one dword per row and 128 k).  One barrier per step, in its middle: the first half
// multiplies what is in registers and reads the second half's fragments; then step t+1
// has landed and everyone is done with stage t, so the second half reads step t+1's
// first fragments and refills stage t with step t+S.  No fragment read waits on the
// barrier it follows, and loads have S - 1/2 steps to arrive.
//
// LDS banks: 16-byte chunks of a row sit at chunk ^ f(row) such that 16 consecutive rows'
// reads of one chunk touch every bank once (64 B rows: (row >> 2) & 3; 128 B rows:
// (row >> 1) & 7; 32 B rows: (row >> 3) & 1).
#include <algorithm>
#include <type_traits>

#include "device_common.h"
#include "mx.h"

namespace moe {

constexpr int kXcd = 8, kBand = 4;
constexpr int kTileN = 256;

typedef int i32x8 __attribute__((ext_vector_type(8)));

// First operand codes `w` with scale byte WB of ws, second `a` with byte AB of as.
template <int BYTE>
__device__ __forceinline__ f32x16 mfma_fp4(u32x4 w, int ws, u32x4 a, int as, f32x16 c) {
  const i32x8 x = {(int)w[0], (int)w[1], (int)w[2], (int)w[3], 0, 0, 0, 0};
  const i32x8 y = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(x, y, c, 4, 4, BYTE, ws, BYTE, as);
}

// global -> LDS from a uniform base and a 32-bit lane offset; the compiler sees no LDS
// write, the kernel waits for vmcnt itself.  dma16: 16 B per lane, dma4: 4 B per lane.
__device__ __forceinline__ void dma16(const void* base, uint32_t off, uint32_t lds_addr) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1"
               :: "v"(off), "s"(base), "s"(lds_addr) : "memory", "m0");
}
__device__ __forceinline__ void dma4(const void* base, uint32_t off, uint32_t lds_addr) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dword %0, %1"
               :: "v"(off), "s"(base), "s"(lds_addr) : "memory", "m0");
}
constexpr int wait_vm(int vm) { return (vm & 0xF) | ((vm >> 4) << 14) | (0x7 << 4) | (0xF << 8); }
constexpr int wait_vm_lgkm0(int vm) { return (vm & 0xF) | ((vm >> 4) << 14) | (0x7 << 4); }

// The experts' rows cut into m-tiles of BM laid end to end; lane l holds experts 4l .. 4l+3.
struct Tiles {
  int lo[4], hi[4], first[4];
  int total;
};

template <int BM>
__device__ __forceinline__ Tiles tiles_of(const int32_t* __restrict__ offsets, int E, int rows) {
  const int lane = __lane_id();
  Tiles t;
  int n[4], sum = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int e = lane * 4 + i;
    t.lo[i] = e < E ? min(max(offsets[e], 0), rows) : 0;
    t.hi[i] = e < E ? min(max(offsets[e + 1], t.lo[i]), rows) : 0;
    n[i] = (t.hi[i] - t.lo[i] + BM - 1) / BM;
    t.first[i] = sum;
    sum += n[i];
  }
  int incl = sum;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int v = __shfl_up(incl, o);
    if (lane >= o) incl += v;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) t.first[i] += incl - sum;
  t.total = __builtin_amdgcn_readfirstlane(__shfl(incl, 63));
  return t;
}

template <int BM>
__device__ __forceinline__ bool find_tile(const Tiles& t, int mt, int& e, int& r0, int& r1) {
  bool found = false;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int n = (t.hi[i] - t.lo[i] + BM - 1) / BM;
    const uint64_t own = __ballot(mt >= t.first[i] && mt < t.first[i] + n);
    if (own) {
      const int l = __builtin_amdgcn_readfirstlane(__ffsll((unsigned long long)own) - 1);
      e = l * 4 + i;
      r0 = __builtin_amdgcn_readfirstlane(__shfl(t.lo[i] + (mt - t.first[i]) * BM, l));
      r1 = min(__builtin_amdgcn_readfirstlane(__shfl(t.hi[i], l)), r0 + BM);
      found = true;
    }
  }
  return found;
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
  const uint8_t* as;       // scales [rows][K/32] (FP4)
  const int32_t* src;      // or null
  int k_top, tokens;
  const int32_t* offsets;
  int E, rows, N, K;
  const uint8_t* w;
  const uint8_t* ws;
  const uint16_t* bias;
  void* out;
};

template <bool FP4, bool UP, int BM>
__global__ __launch_bounds__(256, 1) void mx_tile_kernel(TileArgs p) {
  constexpr int S = FP4 ? 4 : 3;
  constexpr int BK = FP4 ? 128 : 64;
  constexpr int kARow = FP4 ? 64 : 128, kWRow = FP4 ? 64 : 32;   // bytes per row per step
  constexpr int kA = BM * kARow, kW = kTileN * kWRow;
  constexpr int kSA = FP4 ? BM * 4 : 0, kSW = kTileN * 4;
  constexpr int kStage = kA + kW + (FP4 ? 1024 : 0) + kSW;
  constexpr int oW = kA, oSA = kA + kW, oSW = oSA + (FP4 ? 1024 : 0);
  constexpr int kAI = kA / 4096, kWI = kW / 4096;                // 1 KB loads per wave
  constexpr int L = kAI + kWI + (FP4 ? 2 : 1);
  constexpr int kMT = BM / 64, kNT = 4;                          // 32x32 tiles per wave
  static_assert(S * kStage <= 160 * 1024 && kAI >= 1 && kSA <= 1024, "LDS plan");
  __shared__ __attribute__((aligned(1024))) uint8_t lds[S * kStage];

  const int ntn = (p.N + kTileN - 1) / kTileN;
  const Tiles tiles = tiles_of<BM>(p.offsets, p.E, p.rows);
  int mt, nt, e, r0, r1;
  if (!tile_of(tiles.total, ntn, blockIdx.x, mt, nt)) return;
  if (!find_tile<BM>(tiles, mt, e, r0, r1)) return;
  const int n0 = nt * kTileN, N = p.N, K = p.K;

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 1, wn = wave & 1, fr = lane & 31, fc = lane >> 5;

  // ---- load plan: 32-bit lane offsets from uniform bases that advance with k ----
  auto arow = [&](int r) {
    const int g = min(r0 + r, r1 - 1);
    if constexpr (UP) {
      if (p.src) return (int)min((uint32_t)p.src[g] / (uint32_t)p.k_top, (uint32_t)p.tokens - 1u);
    }
    return g;
  };
  const uint32_t a_pitch = FP4 ? K / 2 : K * 2, w_pitch = K / 2, s_pitch = K / 32;
  uint32_t a_off[kAI], w_off[kWI], sa_off = 0, sw_off;
#pragma unroll
  for (int i = 0; i < kAI; ++i) {
    constexpr int kLanes = kARow / 16, kPer = 64 / kLanes;       // lanes per row, rows per load
    const int row = (i * 4 + wave) * kPer + lane / kLanes;
    const int c = (lane % kLanes) ^ (FP4 ? (row >> 2) & 3 : (row >> 1) & 7);
    a_off[i] = (uint32_t)arow(row) * a_pitch + c * 16;
  }
#pragma unroll
  for (int i = 0; i < kWI; ++i) {
    constexpr int kLanes = kWRow / 16, kPer = 64 / kLanes;
    const int row = (i * 4 + wave) * kPer + lane / kLanes;
    const int c = (lane % kLanes) ^ (FP4 ? (row >> 2) & 3 : (row >> 3) & 1);
    w_off[i] = (uint32_t)min(n0 + row, N - 1) * w_pitch + c * 16;
  }
  // Scales: wave w takes rows (64 w + lane) of each operand (BM < 256: some rows twice,
  // with the same value).
  if constexpr (FP4) sa_off = (uint32_t)arow((wave * 64) % BM + lane) * s_pitch;
  sw_off = (uint32_t)min(n0 + wave * 64 + lane, N - 1) * s_pitch;
  const uint8_t* w_base = p.w + (size_t)e * N * (K / 2);
  const uint8_t* ws_base = p.ws + (size_t)e * N * (K / 32);
  const int nk = K / BK;
  const uint32_t lds0 = (uint32_t)(uintptr_t)lds;

  // Load i (0 <= i < L) of step `t` into its stage; steps past the last repeat it (those
  // loads land in a free stage and are never read).
  auto load = [&](int i, int t, int stage) {
    const int s = min(t, nk - 1);
    const uint32_t base = lds0 + stage * kStage;
    if (i < kAI) {
      dma16(p.a + (size_t)s * kARow, a_off[i < kAI ? i : 0], base + (i * 4 + wave) * 1024);
    } else if (i < kAI + kWI) {
      const int j = i - kAI;
      dma16(w_base + (size_t)s * kWRow, w_off[j < 0 || j >= kWI ? 0 : j], base + oW + (j * 4 + wave) * 1024);
    } else if (i == kAI + kWI) {
      dma4(ws_base + (FP4 ? s : s >> 1) * 4, sw_off, base + oSW + wave * 256);
    } else {
      dma4(p.as + s * 4, sa_off, base + oSA + ((wave * 64) % BM) * 4);
    }
  };

  f32x16 acc[kNT][kMT];
#pragma unroll
  for (int j = 0; j < kNT; ++j)
#pragma unroll
    for (int m = 0; m < kMT; ++m)
#pragma unroll
      for (int q = 0; q < 16; ++q) acc[j][m][q] = 0.f;

  auto read_a = [&](int stage, int m, int chunk) {
    const int row = wm * (BM / 2) + m * 32 + fr;
    return ld16(lds + stage * kStage + row * kARow + ((chunk ^ (FP4 ? (row >> 2) & 3 : (row >> 1) & 7)) << 4));
  };
  auto read_w = [&](int stage, int j, int chunk) {
    const int row = wn * 128 + j * 32 + fr;
    return ld16(lds + stage * kStage + oW + row * kWRow + ((chunk ^ (FP4 ? (row >> 2) & 3 : (row >> 3) & 1)) << 4));
  };
  auto read_sa = [&](int stage, int m) {
    const uint32_t v = *reinterpret_cast<const uint32_t*>(lds + stage * kStage + oSA + (wm * (BM / 2) + m * 32 + fr) * 4);
    return (int)(v >> (8 * fc));
  };
  auto read_sw = [&](int stage, int j) {
    return *reinterpret_cast<const uint32_t*>(lds + stage * kStage + oSW + (wn * 128 + j * 32 + fr) * 4);
  };

  // ---- prologue ----
#pragma unroll
  for (int s = 0; s < S; ++s)
#pragma unroll
    for (int i = 0; i < L; ++i) load(i, s, s);
  __builtin_amdgcn_s_waitcnt(wait_vm((S - 1) * L));
  __syncthreads();

  int st = 0;                                          // stage of step t
  if constexpr (FP4) {
    u32x4 xa[kMT], xw[kNT], ya[kMT], yw[kNT];
    int sa[kMT], sw[kNT];
#pragma unroll
    for (int m = 0; m < kMT; ++m) xa[m] = read_a(0, m, fc), sa[m] = read_sa(0, m);
#pragma unroll
    for (int j = 0; j < kNT; ++j) xw[j] = read_w(0, j, fc), sw[j] = (int)(read_sw(0, j) >> (8 * fc));
    constexpr int kM = kMT * kNT;
    for (int t = 0; t < nk; ++t) {
      const int st1 = st == S - 1 ? 0 : st + 1;
      // Slice 0: its MFMAs, reads of slice 1.
#pragma unroll
      for (int q = 0; q < kM; ++q) {
        const int j = q / kMT, m = q % kMT;
        acc[j][m] = mfma_fp4<0>(xw[j], sw[j], xa[m], sa[m], acc[j][m]);
        if (q < kMT) ya[q] = read_a(st, q, 2 + fc);
        if (q < kNT) yw[q] = read_w(st, q, 2 + fc);
        __builtin_amdgcn_sched_barrier(0);
      }
      __builtin_amdgcn_s_waitcnt(wait_vm_lgkm0((S - 2) * L));
      __syncthreads();
      // Slice 1: its MFMAs, reads of the next step's slice 0, loads of step t + S.
      int na[kMT], nw[kNT];
#pragma unroll
      for (int q = 0; q < kM; ++q) {
        const int j = q / kMT, m = q % kMT;
        acc[j][m] = mfma_fp4<2>(yw[j], sw[j], ya[m], sa[m], acc[j][m]);
        if (q < kMT) xa[q] = read_a(st1, q, fc), na[q] = read_sa(st1, q);
        if (q < kNT) xw[q] = read_w(st1, q, fc), nw[q] = (int)(read_sw(st1, q) >> (8 * fc));
#pragma unroll
        for (int i = q * L / kM; i < (q + 1) * L / kM; ++i) load(i, t + S, st);
        __builtin_amdgcn_sched_barrier(0);
      }
#pragma unroll
      for (int m = 0; m < kMT; ++m) sa[m] = na[m];
#pragma unroll
      for (int j = 0; j < kNT; ++j) sw[j] = nw[j];
      st = st1;
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
    auto scale_of = [&](uint32_t v, int t) {
      return __uint_as_float(((v >> (8 * (2 * (t & 1) + fc))) & 0xffu) << 23);
    };
#pragma unroll
    for (int m = 0; m < kMT; ++m) xa[0][m] = read_a(0, m, 4 * fc), xa[1][m] = read_a(0, m, 4 * fc + 1);
#pragma unroll
    for (int j = 0; j < kNT; ++j) raw[j] = read_w(0, j, fc), sc[j] = scale_of(read_sw(0, j), 0);
#pragma unroll
    for (int i = 0; i < 4 * kNT; ++i) widen(raw, sc, wf[0], 0, i);
    constexpr int kM = kMT * kNT;                      // MFMAs per slice
    constexpr int kCv = 4 * kNT;                       // conversions per slice
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
          if (s == 0 && q < kNT) nraw[q] = read_w(st1, q, fc), nsc[q] = scale_of(read_sw(st1, q), t + 1);
          if (s == 0 && q < kMT) xa[0][q] = read_a(st1, q, 4 * fc), xa[1][q] = read_a(st1, q, 4 * fc + 1);
          const int at = s * kM + q;
#pragma unroll
          for (int i = at * L / (2 * kM); i < (at + 1) * L / (2 * kM); ++i) load(i, t + S, st);
          __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
      for (int j = 0; j < kNT; ++j) raw[j] = nraw[j], sc[j] = nsc[j];
      st = st1;
    }
  }
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
  __syncthreads();                                     // LDS free for the epilogue

  // ---- epilogue: each wave turns its sub-tile in LDS and stores whole row segments ----
  constexpr int kOut = UP ? 2 : 4;
  constexpr int kRowB = 128 * kOut, kChunks = kRowB / 16;
  constexpr int kRoom = S * kStage / 4 / kRowB / 32 * 32;         // rows a wave can stage
  constexpr int kPass = kMT * 32 <= kRoom ? kMT * 32 : 32 * (kRoom / 32 >= 2 && kMT % 2 == 0 ? 2 : 1);
  static_assert(kRoom >= 32 && (kMT * 32) % kPass == 0, "epilogue");
  uint8_t* my = lds + wave * kPass * kRowB;
  uint2 braw[kNT][4];
#pragma unroll
  for (int j = 0; j < kNT; ++j)
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const int col = n0 + wn * 128 + j * 32 + 8 * g + 4 * fc;
      braw[j][g] = (p.bias && col < N) ? *reinterpret_cast<const uint2*>(p.bias + (size_t)e * N + col)
                                       : make_uint2(0u, 0u);
    }
#pragma unroll
  for (int pass = 0; pass < kMT * 32 / kPass; ++pass) {
#pragma unroll
    for (int j = 0; j < kNT; ++j)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const float bv[4] = {__uint_as_float(braw[j][g].x << 16), __uint_as_float(braw[j][g].x & 0xffff0000u),
                             __uint_as_float(braw[j][g].y << 16), __uint_as_float(braw[j][g].y & 0xffff0000u)};
#pragma unroll
        for (int i = 0; i < kPass / 32; ++i) {
          const int m = pass * (kPass / 32) + i, row = i * 32 + fr;
          f32x4 v;
#pragma unroll
          for (int q = 0; q < 4; ++q) v[q] = acc[j][m][4 * g + q] + bv[q];
          if constexpr (UP) {
            const int chunk = (j * 4 + g) ^ (row & (kChunks - 1));
            *reinterpret_cast<uint2*>(my + row * kRowB + (chunk << 4) + fc * 8) =
                make_uint2(pack_bf16x2(gelu_erf(v[0]), gelu_erf(v[1])), pack_bf16x2(gelu_erf(v[2]), gelu_erf(v[3])));
          } else {
            const int chunk = (j * 8 + 2 * g + fc) ^ (row & (kChunks - 1));
            *reinterpret_cast<f32x4*>(my + row * kRowB + (chunk << 4)) = v;
          }
        }
      }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_wave_barrier();
    constexpr int kPerInst = 64 / kChunks;
#pragma unroll 4
    for (int rb = 0; rb < kPass; rb += kPerInst) {
      const int row = rb + lane / kChunks, c = lane % kChunks;
      const u32x4 v = ld16(my + row * kRowB + ((c ^ (row & (kChunks - 1))) << 4));
      const int r = r0 + wm * (BM / 2) + pass * kPass + row;
      const int col = n0 + wn * 128 + c * (16 / kOut);
      if (r < r1 && col < N) st16(static_cast<uint8_t*>(p.out) + ((size_t)r * N + col) * kOut, v);
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_wave_barrier();
  }
}

template <bool FP4, bool UP, int BM>
static void launch_tile(const TileArgs& p, hipStream_t s) {
  const long most = p.rows / BM + std::min(p.E, p.rows);           // bound on the m-tiles
  mx_tile_kernel<FP4, UP, BM><<<(unsigned)tile_blocks(most, (p.N + kTileN - 1) / kTileN), 256, 0, s>>>(p);
}

template <bool FP4, bool UP>
static void launch_tile_rows(const TileArgs& p, int bm, hipStream_t s) {
  if (bm == 256) launch_tile<FP4, UP, 256>(p, s);
  else launch_tile<FP4, UP, 128>(p, s);
}

// Rows per tile: 256 from 192 rows per expert on average, else 128.
static int tile_height(long rows, int E) { return rows >= 192L * E ? 256 : 128; }

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
  p.ws = a.ws;
  p.bias = static_cast<const uint16_t*>(a.bias);
  p.out = a.out;
  const int bm = tile_height(p.rows, a.E);
  if (a.fp4) {
    uint8_t* scales = a.act + (size_t)a.a_rows * a.K / 2;
    if (hipError_t e = launch_mx_quantize(a.a, true, a.a_rows, a.K, a.K, a.act, scales, s)) return e;
    p.a = a.act;
    p.as = scales;
    a.up ? launch_tile_rows<true, true>(p, bm, s) : launch_tile_rows<true, false>(p, bm, s);
  } else {
    p.a = static_cast<const uint8_t*>(a.a);
    a.up ? launch_tile_rows<false, true>(p, bm, s) : launch_tile_rows<false, false>(p, bm, s);
  }
  return hipGetLastError();
}

}  // namespace moe
