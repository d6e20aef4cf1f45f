// The shared projection with low-rank adapters, many tokens: LDS-tiled.
//
// Block tile BM tokens x BN columns, 4 waves as 2 x 2, each with BM/2 x BN/2 outputs as 32x32
// MFMA tiles in fp32 accumulators; the MFMA takes W rows as its first operand, so a lane holds
// four consecutive columns of a token.  Steps of 64 k go straight from memory into LDS in whole
// 128-byte lines: two stages of x, three of W, one barrier per step.  A wave that waits to issue
// a load cannot issue MFMAs, so each half step interleaves MFMAs, the LDS reads of the next
// half's fragments and its share of the loads in a fixed order.  Persistent blocks: the loads
// go on into the block's next tile.
//
// At a tile's end the adapters join as further steps of k: for each 32 tokens of a wave and each
// different adapter a among them, B_a (its rows as they lie in memory: 16 bytes are 8 ranks of a
// column) times u, which the first kernel left as bf16 terms (two under a bf16 result, 17 bits;
// three under fp32, all of its 24).  Where the 32 tokens have several adapters u is 0 for all
// but a's own.  What of B_a is infinite or NaN goes by a product of its own, with u's sign
// (1, -1 or 0) in one term: 0 times it would spread to the others, and u's later terms, 0 or of
// either sign, would make NaN of an infinity.  In the main product +-1 stands in its place, so that an
// infinite u does not meet a 0.
//
// 16384 x 4096 -> 14336, rank 16, GELU: 1520 to 1580 us, 1.25 PFLOP/s (1.50 in a library product of
// 16384 x 16384 x 8192): steps 1335, GELU 130, stores 60, adapters 40.  8192 x 2816 -> 2048, rank 32,
// fp32: 88 to 92 us, one tile a CU.
//
// LDS: rows of 128 B, the eight 16-byte chunks of row r at chunk ^ ((r >> 1) & 7): a fragment
// read (16 rows, one chunk) touches every bank once.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "device_common.h"
#include "lora.h"
#include "lora_parts.h"

namespace moe {

constexpr int kLoraXcds = 8, kLoraBand = 4, kLoraCus = 256;

// Tile of block b.  Whole groups of 32 m-tiles: XCD b % 8 owns 4 of them and walks them n-tile by
// n-tile, so the blocks it runs together share their tokens in its L2 and all XCDs sweep the
// same columns of W.  The m-tiles left over go in bands of 8, each n-tile by n-tile, and every XCD
// takes one run of that order: with few tokens each W tile is read into one L2 (dealt round-robin,
// 512 tokens, 4096 -> 14336: 124 us instead of 83).
__device__ __forceinline__ bool lora_tile_of(int total, int ntn, int b, int& mt, int& nt) {
  constexpr int kGroup = kLoraXcds * kLoraBand, kRest = 8;
  const int x = b % kLoraXcds, i = b / kLoraXcds;
  const int G = total / kGroup, full = G * kLoraBand * ntn, lm = total - G * kGroup;
  if (i < full) {
    const int g = i / (kLoraBand * ntn), rem = i - g * kLoraBand * ntn;
    nt = rem / kLoraBand;
    mt = g * kGroup + x * kLoraBand + rem % kLoraBand;
    return true;
  }
  const int run = (lm * ntn + kLoraXcds - 1) / kLoraXcds, j = i - full, v = x * run + j;
  if (j >= run || v >= lm * ntn) return false;
  const int band = v / (kRest * ntn), rem = v - band * kRest * ntn, wide = min(kRest, lm - band * kRest);
  nt = rem / wide;
  mt = G * kGroup + band * kRest + rem % wide;
  return true;
}

static long lora_tile_blocks(long total, long ntn) {
  const long G = total / (kLoraXcds * kLoraBand), lm = total % (kLoraXcds * kLoraBand);
  return kLoraXcds * (G * kLoraBand * ntn + (lm * ntn + kLoraXcds - 1) / kLoraXcds);
}

// Whether the lower or upper bf16 of a word is infinite or NaN.
__device__ __forceinline__ bool infinite_lo(uint32_t w) { return (w & 0x7f80u) == 0x7f80u; }
__device__ __forceinline__ bool infinite_hi(uint32_t w) { return (w & 0x7f800000u) == 0x7f800000u; }

// Of two bf16 the signs: 1, -1 or 0.
constexpr uint32_t kSigns = 0x80008000u, kOnes = 0x3f803f80u;
__device__ __forceinline__ uint32_t signs_of(uint32_t w) {
  const uint32_t some = ((w & 0x7fffu) ? 0xffffu : 0u) | ((w & 0x7fff0000u) ? 0xffff0000u : 0u);
  return (w & kSigns) | (kOnes & some);
}

// Of two pairs of 16 bits the larger of each half.
__device__ __forceinline__ uint32_t max_pair(uint32_t a, uint32_t b) {
  typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, a), __builtin_bit_cast(u16x2, b)));
}

// TERMS: the bf16 terms of u, 2 for a bf16 result, 3 for fp32; 0: a part of the k range of W x, or
// of A x as further columns, stored in fp32 for a finish of its own (one tile a block).
// AS: stages of x; W has one more.
template <int BM, int BN, int TERMS, int AS, int OCC>
__global__ __launch_bounds__(256, OCC) void lora_tile_kernel(LoraPartArgs all) {
  const LoraArgs& p = all.a;
  constexpr int kA = BM * 128, kW = BN * 128, kWS = AS + 1;        // bytes a stage; stages of W
  constexpr int oW = AS * kA;
  constexpr int kMT = BM / 64, kNT = BN / 64;                      // 32x32 tiles per wave
  constexpr int kAI = BM / 32, kWI = BN / 32;                      // 1 KB loads per wave
  constexpr bool F32 = TERMS == 3, PART = TERMS == 0;
  // Loads that may be under way when the next step's have to be there (see the loop).
  constexpr int kUnderWay = (AS - 1) * kWI + (AS - 2) * kAI;
  static_assert(OCC * (AS * kA + kWS * kW) <= 160 * 1024 && (AS - 1) * (kWI + kAI) < 64, "LDS plan");
  __shared__ __attribute__((aligned(1024))) uint8_t lds[AS * kA + kWS * kW];

  const int T = p.sh.T, N = p.sh.n, K = p.sh.d, nk = K / 64;
  const int ntn = (N + BN - 1) / BN, total = (T + BM - 1) / BM;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 1, wn = wave & 1, fr = lane & 31, fc = lane >> 5;
  const uint32_t lds0 = (uint32_t)(uintptr_t)lds;

  struct Where {
    int r0, n0;
  };
  // A part: which of the k range, and of which columns.
  LoraUnit unit;
  int groups = 0, wide[kWI];                           // groups of 16 ranks; the ids that the wave loads
  if constexpr (PART) {
    if (!lora_unit<BM, BN>(all, unit)) return;
    if (unit.of_a) {
      int* list = reinterpret_cast<int*>(lds);
      groups = lora_list<BM>(p, unit.t0, list) * (lora_pitch(p.sh.rank) / 16);
      if (unit.g0 >= groups) return;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < kWI; ++i)
        wide[i] = __builtin_amdgcn_readfirstlane(list[min(unit.g0 + (i * 4 + wave) / 2, groups - 1) / (lora_pitch(p.sh.rank) / 16)]);
      __syncthreads();
    }
  }
  const int k0 = PART ? unit.k0 : 0, k1 = PART ? unit.k1 : nk;
  int b = blockIdx.x;
  auto locate = [&](Where& w) {
    int mt, nt;
    if (!lora_tile_of(total, ntn, b, mt, nt)) return false;
    w = Where{mt * BM, nt * BN};
    return true;
  };
  // Loads: instruction i of a wave fills rows (4 i + wave) 8 + lane / 8.  32-bit lane offsets
  // (x and W are under 4 GiB) from uniform bases; rows past the end read the last.
  uint32_t a_off[kAI], w_off[kWI];
  auto row_of = [&](int i) { return (i * 4 + wave) * 8 + (lane >> 3); };
  auto chunk_of = [&](int row) { return (uint32_t)(((lane & 7) ^ ((row >> 1) & 7)) << 4); };
  auto aim_a = [&](const Where& w) {
#pragma unroll
    for (int i = 0; i < kAI; ++i) a_off[i] = (uint32_t)min(w.r0 + row_of(i), T - 1) * (uint32_t)K * 2u + chunk_of(row_of(i));
  };
  const uint8_t *xb = reinterpret_cast<const uint8_t*>(p.x), *wb[PART ? kWI : 1];
  wb[0] = reinterpret_cast<const uint8_t*>(p.w);
  auto aim_w = [&](const Where& w) {
#pragma unroll
    for (int i = 0; i < kWI; ++i) {
      if (PART && unit.of_a) {                         // rows of one adapter in every load
        const int rank = p.sh.rank, g = min(unit.g0 + (i * 4 + wave) / 2, groups - 1);
        const int row = min(g % (lora_pitch(rank) / 16) * 16 + row_of(i) % 16, rank - 1);
        wb[PART ? i : 0] = reinterpret_cast<const uint8_t*>(p.a) + (size_t)wide[i] * rank * K * 2;
        w_off[i] = (uint32_t)row * (uint32_t)K * 2u + chunk_of(row_of(i));
      } else {
        if (PART) wb[PART ? i : 0] = reinterpret_cast<const uint8_t*>(p.w);
        w_off[i] = (uint32_t)min(w.n0 + row_of(i), N - 1) * (uint32_t)K * 2u + chunk_of(row_of(i));
      }
    }
  };
  auto load_a = [&](int i, int stage, int step) {
    dma16(xb + (size_t)step * 128, a_off[i], lds0 + stage * kA + (i * 4 + wave) * 1024);
  };
  auto load_w = [&](int i, int stage, int step) {
    dma16(wb[PART ? i : 0] + (size_t)step * 128, w_off[i], lds0 + oW + stage * kW + (i * 4 + wave) * 1024);
  };

  Where cur, next;
  if (PART) cur = Where{unit.t0, unit.n0};
  else if (!locate(cur)) return;
  next = cur;
  bool more = !PART;
  aim_a(cur);
  aim_w(cur);
  int as = k0, ws = k0;                                // the steps to load next
  // After a step's loads of W: on to the next step, or tile.  The loads of x follow half a step
  // later, with the tile found here.  Past the last tile the last step is loaded again, unread.
  bool a_moves = false;
  auto advance_w = [&]() {
    if (++ws < k1) return;
    if (more) {
      b += gridDim.x;
      Where w;
      more = locate(w);
      if (more) {
        next = w;
        aim_w(w);
        ws = 0;
        a_moves = true;
        return;
      }
    }
    ws = k1 - 1;
  };
  auto advance_a = [&]() {
    if (++as < k1) return;
    if (a_moves) {
      aim_a(next);
      as = 0;
      a_moves = false;
      return;
    }
    as = k1 - 1;
  };

  f32x16 acc[kNT][kMT];
  // The large tile's accumulators fill the matrix cores' registers: held there, or the compiler
  // moves some in and out in every step, and all of them at once, by spilling, at the end.
  auto pin_one = [&](int j, int m) {
    if constexpr (BM * BN >= 256 * 256) asm volatile("" : "+a"(acc[j][m]));
  };
  auto pin = [&]() {
#pragma unroll
    for (int j = 0; j < kNT; ++j)
#pragma unroll
      for (int m = 0; m < kMT; ++m) pin_one(j, m);
  };
  constexpr int kReads = 2 * (kMT + kNT), kMfmas = 2 * kMT * kNT;  // per half step
  constexpr int kPer = 2;                              // reads behind one MFMA, until all are done
  static_assert(kPer * kMfmas >= kReads, "reads");
  u32x4 xa[2][kMT], xw[2][kNT], ya[2][kMT], yw[2][kNT];
  // Fragment addresses: rows 32 apart share their swizzle.
  const uint32_t swz = (fr >> 1) & 7;
  const uint32_t a_lane = (uint32_t)(wm * (BM / 2) + fr) * 128, w_lane = oW + (uint32_t)(wn * (BN / 2) + fr) * 128;
  auto read_at = [&](u32x4 (&fa)[2][kMT], u32x4 (&fw)[2][kNT], int sa, int sw, int half, int r) {
    const int sl = r / (kMT + kNT), q = r % (kMT + kNT);
    const uint32_t c = (((half * 2 + sl) * 2 + fc) ^ swz) << 4;
    if (q < kMT) fa[sl][q] = ld16(lds + (sa * kA + a_lane + c) + q * 4096);
    else fw[sl][q - kMT] = ld16(lds + (sw * kW + w_lane + c) + (q - kMT) * 4096);
  };
  auto half_step = [&](const u32x4 (&fa)[2][kMT], const u32x4 (&fw)[2][kNT], u32x4 (&na)[2][kMT],
                       u32x4 (&nw)[2][kNT], int sa, int sw, int half, auto load_fn, auto loads) {
    constexpr int L = decltype(loads)::value;
#pragma unroll
    for (int m = 0; m < kMfmas; ++m) {
      const int sl = m / (kMT * kNT), j = m / kMT % kNT, i = m % kMT;
      acc[j][i] = mfma32_bf16(fw[sl][j], fa[sl][i], acc[j][i]);
#pragma unroll
      for (int r = m * kPer; r < (m + 1) * kPer; ++r)
        if (r < kReads) read_at(na, nw, sa, sw, half, r);
#pragma unroll
      for (int q = m * L / kMfmas; q < (m + 1) * L / kMfmas; ++q) load_fn(q);
      __builtin_amdgcn_sched_barrier(0);
    }
  };

  // The adapters of the tile's tokens, lane l that of row 32 m + l % 32 of the wave (-1: none;
  // rows past the end take their neighbours').
  int ids[kMT];
  auto load_ids = [&](const Where& w) {
#pragma unroll
    for (int m = 0; m < kMT; ++m) {
      const int id = p.adapter[min(w.r0 + wm * (BM / 2) + m * 32 + fr, T - 1)];
      ids[m] = (uint32_t)id < (uint32_t)p.sh.N ? id : -1;
    }
  };
  const int rank = p.sh.rank, pitch = (rank + 15) / 16 * 16;
  auto expand = [&](const Where& w) {
    constexpr int kTerms = PART ? 1 : TERMS;
    const uint16_t* u = static_cast<const uint16_t*>(p.u);
#pragma unroll
    for (int m = 0; m < kMT; ++m) {
      const uint16_t* um = u + (size_t)min(w.r0 + wm * (BM / 2) + m * 32 + fr, T - 1) * pitch + fc * 8;
      uint64_t left = __ballot(ids[m] >= 0);
      while (left) {
        const int id = __builtin_amdgcn_readlane(ids[m], __ffsll((unsigned long long)left) - 1);
        const uint64_t same = __ballot(ids[m] == id);
        left &= ~same;
        const bool mine = ids[m] == id;
        for (int k = 0; k < pitch; k += 16) {
          u32x4 bf[kNT], uf[kTerms];
#pragma unroll
          for (int j = 0; j < kNT; ++j) {
            const int col = min(w.n0 + wn * (BN / 2) + j * 32 + fr, N - 1);
            const bool in = k + fc * 8 < rank;             // rank 8 more than a multiple of 16
            bf[j] = in ? ld16(p.b + ((size_t)id * N + col) * rank + k + fc * 8) : u32x4{0, 0, 0, 0};
          }
#pragma unroll
          for (int q = 0; q < kTerms; ++q) {
            uf[q] = ld16(um + (size_t)q * T * pitch + k);
            uf[q] = mine ? uf[q] : u32x4{0, 0, 0, 0};
          }
          uint32_t most = 0;
#pragma unroll
          for (int j = 0; j < kNT; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) most = max_pair(most, bf[j][i] & ~kSigns);
          if (__ballot(infinite_lo(most) | infinite_hi(most))) {   // a few registers of the 256 x 256 tile spill for it, outside the steps
            u32x4 sign;
#pragma unroll
            for (int i = 0; i < 4; ++i) sign[i] = signs_of(uf[0][i]);
#pragma unroll
            for (int j = 0; j < kNT; ++j) {
              u32x4 far;
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const uint32_t v = bf[j][i], bad = (infinite_lo(v) ? 0xffffu : 0u) | (infinite_hi(v) ? 0xffff0000u : 0u);
                far[i] = v & bad;
                bf[j][i] = (v & (~bad | kSigns)) | (kOnes & bad);
              }
              f32x16 v = {};
              v = mfma32_bf16(far, sign, v);
#pragma unroll
              for (int i = 0; i < 16; ++i) acc[j][m][i] += mine ? v[i] : 0.f;
              pin_one(j, m);
            }
          }
#pragma unroll
          for (int j = 0; j < kNT; ++j)
#pragma unroll
            for (int q = 0; q < kTerms; ++q) acc[j][m] = mfma32_bf16(bf[j], uf[q], acc[j][m]);
        }
      }
    }
  };

  // Bias, GELU, stores straight from the accumulators.  A lane has columns 8 g + 4 fc .. + 3 of
  // its token; bf16 first swaps between the lane halves, so that one has all 8 columns of g and
  // the other those of g + 1.
  auto finish = [&](const Where& w) {
#pragma unroll
    for (int j = 0; j < kNT; ++j) {
      const int col0 = w.n0 + wn * (BN / 2) + j * 32;
      uint2 braw[4];
#pragma unroll
      for (int g = 0; g < 4; ++g)
        braw[g] = (p.bias && col0 < N) ? *reinterpret_cast<const uint2*>(p.bias + col0 + 8 * g + 4 * fc) : make_uint2(0u, 0u);
#pragma unroll
      for (int m = 0; m < kMT; ++m) {
        const int r = w.r0 + wm * (BM / 2) + m * 32 + fr;
        const bool in = r < T && col0 < N;
        pin_one(j, m);
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
        if (p.sh.gelu) {
#pragma unroll
          for (int g = 0; g < 4; ++g)
#pragma unroll
            for (int q = 0; q < 4; ++q) v[g][q] = F32 ? gelu_f32(v[g][q]) : gelu_for_bf16(v[g][q]);
        }
        if constexpr (F32) {
          float* o = static_cast<float*>(p.y) + (size_t)r * N + col0 + 4 * fc;
#pragma unroll
          for (int g = 0; g < 4; ++g)
            if (in) *reinterpret_cast<f32x4*>(o + 8 * g) = v[g];
        } else {
          uint16_t* o = static_cast<uint16_t*>(p.y) + (size_t)r * N + col0 + 8 * fc;
#pragma unroll
          for (int g = 0; g < 4; g += 2) {
            uint32_t h[2][2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              h[i][0] = pack_bf16x2(v[g + i][0], v[g + i][1]);
              h[i][1] = pack_bf16x2(v[g + i][2], v[g + i][3]);
            }
            const auto s0 = __builtin_amdgcn_permlane32_swap(h[0][0], h[1][0], false, false);
            const auto s1 = __builtin_amdgcn_permlane32_swap(h[0][1], h[1][1], false, false);
            if (in) st16(o + 8 * g, u32x4{s0[0], s1[0], s0[1], s1[1]});
          }
        }
      }
    }
  };

  // Step t: its x in stage t % AS, its W in t % (AS + 1).  First half: MFMAs of the fragments at
  // hand, reads of the step's second half, loads of W AS steps on (into the stage of step t - 1,
  // which nobody reads any more).  Then the next step's x and W have landed, all but the AS - 1
  // loads of W and AS - 2 of x after them; barrier.  Second half: reads of the next step's
  // first half, loads of x AS steps on (every wave is done with this stage).
#pragma unroll
  for (int s = 0; s < AS; ++s) {
#pragma unroll
    for (int i = 0; i < kWI; ++i) load_w(i, s, ws);
    advance_w();
#pragma unroll
    for (int i = 0; i < kAI; ++i) load_a(i, s, as);
    advance_a();
  }
  __builtin_amdgcn_s_waitcnt(wait_vm((AS - 1) * (kWI + kAI)));
  __syncthreads();
#pragma unroll
  for (int r = 0; r < kReads; ++r) read_at(xa, xw, 0, 0, 0, r);
  int sa = 0, sw = 0;
  using LoadsA = std::integral_constant<int, kAI>;
  using LoadsW = std::integral_constant<int, kWI>;
  for (;;) {
#pragma unroll
    for (int j = 0; j < kNT; ++j)
#pragma unroll
      for (int m = 0; m < kMT; ++m)
#pragma unroll
        for (int q = 0; q < 16; ++q) acc[j][m][q] = 0.f;
    const Where done = cur;
    bool go_on = false;
    if constexpr (!PART) load_ids(cur);
    for (int t = k0; t < k1; ++t) {
      pin();
      const int sw1 = sw == AS ? 0 : sw + 1, sw2 = sw == 0 ? AS : sw - 1, sa1 = sa == AS - 1 ? 0 : sa + 1;
      half_step(xa, xw, ya, yw, sa, sw, 1, [&](int i) { load_w(i, sw2, ws); }, LoadsW{});
      advance_w();
      __builtin_amdgcn_s_waitcnt(wait_vm_lgkm0(kUnderWay));
      __syncthreads();
      half_step(ya, yw, xa, xw, sa1, sw1, 0, [&](int i) { load_a(i, sa, as); }, LoadsA{});
      advance_a();
      sa = sa1;
      sw = sw1;
    }
    if constexpr (PART) break;
    go_on = next.r0 != cur.r0 || next.n0 != cur.n0;
    expand(done);
    finish(done);
    if (!go_on) break;
    cur = next;
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");       // no load outlives its LDS
  if constexpr (PART) {
    // A lane has columns 8 g + 4 fc .. + 3 of token fr: of W, or of its own adapter's ranks.
    const int per = pitch / 16;
    int* list = reinterpret_cast<int*>(lds);
    if (unit.of_a) {
      __syncthreads();
      lora_list<BM>(p, unit.t0, list);
      __syncthreads();
    }
#pragma unroll
    for (int m = 0; m < kMT; ++m) {
      const int t = unit.t0 + wm * (BM / 2) + m * 32 + fr;
      const int id = unit.of_a && t < T ? p.adapter[t] : -1;
#pragma unroll
      for (int j = 0; j < kNT; ++j)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const int c = wn * (BN / 2) + j * 32 + 8 * g + 4 * fc;
          f32x4 v;
#pragma unroll
          for (int q = 0; q < 4; ++q) v[q] = acc[j][m][4 * g + q];
          if (!unit.of_a) {
            if (t < T && unit.n0 + c < N)
              *reinterpret_cast<f32x4*>(all.part + ((size_t)unit.split * T + t) * N + unit.n0 + c) = v;
          } else {
            const int group = unit.g0 + c / 16, r = group % per * 16 + c % 16;
            if (t >= T || group >= groups || id != list[group / per]) continue;
#pragma unroll
            for (int q = 0; q < 4; ++q) v[q] = r + q < rank ? v[q] : 0.f;
            *reinterpret_cast<f32x4*>(all.u + ((size_t)unit.split * T + t) * pitch + r) = v;
          }
        }
    }
  }
}

void launch_lora_part_tile(const LoraPartArgs& p, unsigned grid, hipStream_t s) {
  lora_tile_kernel<128, 128, 0, 2, 2><<<grid, 256, 0, s>>>(p);
}

template <int BM, int BN, int OCC>
static void run_tile(const LoraArgs& a, hipStream_t s) {
  const long blocks = lora_tile_blocks((a.sh.T + BM - 1) / BM, (a.sh.n + BN - 1) / BN);
  const unsigned grid = (unsigned)std::min(blocks, (long)kLoraCus * OCC);
  const LoraPartArgs p{a, 1, 0, nullptr, nullptr};
  if (a.sh.f32_out) lora_tile_kernel<BM, BN, 3, 2, OCC><<<grid, 256, 0, s>>>(p);
  else lora_tile_kernel<BM, BN, 2, 2, OCC><<<grid, 256, 0, s>>>(p);
}

// Large tiles once they fill three quarters of the CUs (16384 tokens, 4096 -> 14336: 1557 us, small ones
// 2049); before that small ones, two a CU.
hipError_t launch_lora_tile(const LoraArgs& a, hipStream_t s) {
  const long big = (long)((a.sh.T + 255) / 256) * ((a.sh.n + 255) / 256);
  if (big >= 192) run_tile<256, 256, 1>(a, s);
  else run_tile<128, 128, 2>(a, s);
  return hipGetLastError();
}

}  // namespace moe
