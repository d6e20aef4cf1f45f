// A projection shared by all tokens, with a low-rank adapter of each token's own beside it:
//   y_t = act(W x_t + bias + scale_a B_a (A_a x_t)),  a = adapter[t]; outside [0, N): no adapter
//
// The tokens stay in their order.  A tile of tokens runs once through the list of the different
// adapters that its tokens have: one for a long request, as many as tokens in a decode batch.
// Three ways: one token (lora_token_kernel), up to some hundred (lora_part_kernel and
// lora_finish_kernel), more (lora_shrink_kernel, then the tiles of lora_tile.hip).
#include <algorithm>
#include <type_traits>

#include "device_common.h"
#include "lora.h"

namespace moe {

// Fragments of `NA` and `NB` 16-row groups, 32 values of k each, through U register stages; the
// WAVES waves of a block take every WAVES-th step of k.  acc[j][m] += A_j B_m^T.
template <int NA, int NB, int U, int WAVES>
__device__ __forceinline__ void dot_rows(const uint16_t* (&pa)[NA], const uint16_t* (&pb)[NB], int steps, int wave,
                                         f32x4 (&acc)[NA][NB]) {
  u32x4 fa[U][NA], fb[U][NB];
  const int mine = (steps - wave + WAVES - 1) / WAVES, last = steps - 1;
  auto load = [&](int slot, int i) {                 // past the end: the last step again, not used
    const int k = min(wave + i * WAVES, last) * 32;
#pragma unroll
    for (int j = 0; j < NA; ++j) fa[slot][j] = ld16(pa[j] + k);
#pragma unroll
    for (int m = 0; m < NB; ++m) fb[slot][m] = ld16(pb[m] + k);
  };
  auto multiply = [&](int slot) {
#pragma unroll
    for (int j = 0; j < NA; ++j)
#pragma unroll
      for (int m = 0; m < NB; ++m) acc[j][m] = mfma_bf16(fa[slot][j], fb[slot][m], acc[j][m]);
  };
#pragma unroll
  for (int q = 0; q < U; ++q) load(q, q);
  int i = 0;
  for (; i + U <= mine; i += U) {
#pragma unroll
    for (int q = 0; q < U; ++q) {
      multiply(q);
      load(q, i + U + q);
    }
  }
#pragma unroll
  for (int q = 0; q < U; ++q)
    if (i + q < mine) multiply(q);
}

// ---------------------------------------------------------------------------
// u = scale A x before the tiled product, as bf16 terms: a block has 16 MT tokens and first lists
// the different adapters among them.  An adapter is pitch / 16 groups of 16 ranks; a pass over
// k takes NS groups, of one adapter or of several, so that x is read once for a few
// adapters.  The waves share out k, so the sums meet in LDS.  Bound by reading x.
// ---------------------------------------------------------------------------
template <int MT, int NS, int WAVES>
__global__ __launch_bounds__(WAVES * 64) void lora_shrink_kernel(LoraArgs a) {
  constexpr int kRows = 16 * MT, kRanks = 16 * NS;
  __shared__ __attribute__((aligned(16))) float part[WAVES][kRows][kRanks];
  __shared__ int list[kRows];
  const int T = a.sh.T, d = a.sh.d, rank = a.sh.rank, pitch = (rank + 15) / 16 * 16, per = pitch / 16;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int fr = lane & 15, fc = lane >> 4, t0 = blockIdx.x * kRows;
  const int own = t0 + lane < T && lane < kRows ? a.adapter[t0 + lane] : -1;   // lane l: token t0 + l
  int count = 0;
  for (uint64_t left = __ballot((uint32_t)own < (uint32_t)a.sh.N); left; ++count) {
    const int id = __builtin_amdgcn_readlane(own, __ffsll((unsigned long long)left) - 1);
    left &= ~__ballot(own == id);
    if (threadIdx.x == 0) list[count] = id;
  }
  __syncthreads();
  const uint16_t* px[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) px[m] = a.x + (size_t)min(t0 + m * 16 + fr, T - 1) * d + fc * 8;
  const int groups = count * per;
  for (int g0 = 0; g0 < groups; g0 += NS) {
    const uint16_t* pa[NS];
#pragma unroll
    for (int j = 0; j < NS; ++j) {
      const int g = min(g0 + j, groups - 1);
      pa[j] = a.a + ((size_t)list[g / per] * rank + min(g % per * 16 + fr, rank - 1)) * d + fc * 8;
    }
    f32x4 acc[NS][MT] = {};
    dot_rows<NS, MT, (NS + MT >= 8 ? 2 : NS + MT >= 4 ? 4 : 8), WAVES>(pa, px, d / 32, wave, acc);
    // A lane has ranks 4 fc .. + 3 of token fr.
#pragma unroll
    for (int j = 0; j < NS; ++j)
#pragma unroll
      for (int m = 0; m < MT; ++m)
        *reinterpret_cast<f32x4*>(&part[wave][m * 16 + fr][j * 16 + fc * 4]) = acc[j][m];
    __syncthreads();
    for (int o = threadIdx.x; o < kRows * kRanks / 2; o += WAVES * 64) {   // two ranks a thread
      const int row = o / (kRanks / 2), r = o % (kRanks / 2) * 2, g = g0 + r / 16, t = t0 + row;
      if (t >= T || g >= groups) continue;
      const int id = list[g / per], at_rank = g % per * 16 + r % 16;
      if (a.adapter[t] != id) continue;
      float v[2] = {0.f, 0.f};
#pragma unroll
      for (int w = 0; w < WAVES; ++w) v[0] += part[w][row][r], v[1] += part[w][row][r + 1];
      const float scale = a.scale ? a.scale[id] : 1.f;
#pragma unroll
      for (int q = 0; q < 2; ++q) v[q] = at_rank + q < rank ? v[q] * scale : 0.f;
      const size_t at = (size_t)t * pitch + at_rank;
      uint16_t* u = static_cast<uint16_t*>(a.u);
      const int terms = a.sh.f32_out ? 3 : 2;
      for (int q = 0; q < terms; ++q) {
        const uint32_t h = pack_bf16x2(v[0], v[1]);
        *reinterpret_cast<uint32_t*>(u + (size_t)q * T * pitch + at) = h;
        // what the term left over; nothing of an infinity
        v[0] = (h & 0x7f80u) == 0x7f80u ? 0.f : v[0] - __uint_as_float(h << 16);
        v[1] = (h & 0x7f800000u) == 0x7f800000u ? 0.f : v[1] - __uint_as_float(h & 0xffff0000u);
      }
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------
// One token: bound by the bytes of W.  A block has 16 NNT columns; its adapter's 16 RANKS ranks are
// further rows beside them, so every block has u itself and one launch does all; A is read from
// memory once and then from L2.  Eight waves share out k, fragments go straight from memory to
// registers, the sums meet in LDS, where a thread finishes a column.
// ---------------------------------------------------------------------------
constexpr int kWaves = 8;

// Eight ranks of B times eight values of u.
__device__ __forceinline__ float dot8(const u32x4& q, const float* u, float s) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    s = fmaf(__uint_as_float(q[i] << 16), u[2 * i], s);
    s = fmaf(__uint_as_float(q[i] & 0xffff0000u), u[2 * i + 1], s);
  }
  return s;
}

template <int NNT, int RANKS>
__global__ __launch_bounds__(kWaves * 64) void lora_token_kernel(LoraArgs a) {
  constexpr int kCols = 16 * NNT, NA = NNT + RANKS;
  __shared__ __attribute__((aligned(16))) float part[kWaves][16 * NA];
  __shared__ __attribute__((aligned(16))) float su[16 * RANKS];
  const int d = a.sh.d, n = a.sh.n, rank = a.sh.rank;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int fr = lane & 15, fc = lane >> 4, n0 = blockIdx.x * kCols;
  const int given = a.adapter[0], id = (uint32_t)given < (uint32_t)a.sh.N ? given : -1;
  const int any = max(id, 0);                          // without an adapter A and B are read, not used
  const uint16_t *px[1] = {a.x + fc * 8}, *pw[NA];
#pragma unroll
  for (int j = 0; j < NNT; ++j) pw[j] = a.w + (size_t)min(n0 + j * 16 + fr, n - 1) * d + fc * 8;
#pragma unroll
  for (int j = 0; j < RANKS; ++j) pw[NNT + j] = a.a + ((size_t)any * rank + min(j * 16 + fr, rank - 1)) * d + fc * 8;
  // The thread's column (its first 16 ranks of B), scale and bias, under way with the rest.
  const int c = min(n0 + (int)threadIdx.x, n - 1);
  u32x4 qb[2] = {};
  float bias = 0.f, scale = 1.f;
  if (threadIdx.x < kCols) {
    const uint16_t* b = a.b + ((size_t)any * n + c) * rank;
    qb[0] = ld16(b);
    if (rank > 8) qb[1] = ld16(b + 8);
    if (a.bias) bias = bf16_to_f32(a.bias[c]);
  }
  if (a.scale) scale = a.scale[any];
  f32x4 acc[NA][1] = {};
  dot_rows<NA, 1, (NA >= 5 ? 4 : NA >= 3 ? 8 : 12), kWaves>(pw, px, d / 32, wave, acc);
  // Every token of the tile is the same one: lane fr = 0 has columns 4 fc .. + 3.
  if (fr == 0)
#pragma unroll
    for (int j = 0; j < NA; ++j) *reinterpret_cast<f32x4*>(&part[wave][j * 16 + fc * 4]) = acc[j][0];
  __syncthreads();
  auto sum = [&](int i) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) v += part[w][i];
    return v;
  };
  // The last wave sums u, the first columns' threads what they wait for anyway.
  if ((int)threadIdx.x >= kWaves * 64 - 16 * RANKS) {
    const int r = threadIdx.x - (kWaves * 64 - 16 * RANKS);
    su[r] = r < rank ? sum(kCols + r) * scale : 0.f;
  }
  float v = threadIdx.x < kCols ? sum(threadIdx.x) + bias : 0.f;
  __syncthreads();
  if (threadIdx.x >= kCols || n0 + (int)threadIdx.x >= n) return;
  if (id >= 0) {
    float s = dot8(qb[0], su, 0.f);
    if (rank > 8) s = dot8(qb[1], su + 8, s);
    for (int r = 16; r < rank; r += 8) s = dot8(ld16(a.b + ((size_t)id * n + c) * rank + r), su + r, s);
    v += s;
  }
  if (a.sh.f32_out) static_cast<float*>(a.y)[c] = a.sh.gelu ? gelu_erf(v) : v;
  else static_cast<uint16_t*>(a.y)[c] = (uint16_t)pack_bf16x2(a.sh.gelu ? gelu_for_bf16(v) : v, 0.f);
}

// ---------------------------------------------------------------------------
// Up to some hundred tokens: the bytes of W bound it, and the latency of what has to wait for
// what.  So W x and A x go in one kernel, as columns of one product: a block has BM tokens
// and 64 columns, of W or of the adapters that its tokens have (16 ranks of one after the other's),
// and one part of k.  It stores fp32 sums, of A x a token's own adapter's only.  A second kernel
// adds up the parts, B u, the bias and the activation.
//
// Both operands go from memory into LDS in runs of RB bytes of every row, ST stages, the
// 16-byte pieces of row r at piece ^ swizzle(r) so that 16 rows' reads of one piece touch every
// bank once.  Four waves as WM x 4 / WM.  Two blocks fit a CU, so one's start and end go under
// the other's loads.
// ---------------------------------------------------------------------------
struct PartArgs {
  LoraArgs a;
  int splits, a_tiles;                 // parts of k; column tiles that A can have per BM tokens
  float* part;                         // [splits][T][n]
  float* u;                            // [splits][T][pitch]
};

constexpr int kPartCols = 64;

template <int BM, int RB, int ST, int WM>
__global__ __launch_bounds__(256, 2) void lora_part_kernel(PartArgs p) {
  constexpr int kPieces = RB / 16, kPer = 1024 / RB;             // of a row; rows per load
  constexpr int kA = BM * RB, kStage = (BM + kPartCols) * RB;
  constexpr int kAI = kA / 4096, kWI = kPartCols * RB / 4096, L = kAI + kWI;   // loads per wave
  constexpr int kM = BM / WM / 16, kN = kPartCols * WM / 64;     // 16x16 tiles per wave
  static_assert(kA % 4096 == 0 && 2 * (ST * kStage + BM * 8 + 64) <= 160 * 1024, "LDS plan");
  __shared__ __attribute__((aligned(1024))) uint8_t lds[ST * kStage];
  __shared__ int ids[BM], list[BM];
  const LoraArgs& a = p.a;
  const int T = a.sh.T, d = a.sh.d, n = a.sh.n, rank = a.sh.rank, pitch = (rank + 15) / 16 * 16, per = pitch / 16;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int fr = lane & 15, fc = lane >> 4, wm = wave % WM, wn = wave / WM;
  const uint32_t lds0 = (uint32_t)(uintptr_t)lds;

  // Block b: the row tiles of one (column tile, part of k) follow one another on one XCD.
  const int mts = (T + BM - 1) / BM, cols = n / kPartCols + p.a_tiles;
  const int q = blockIdx.x / 8, cs = q / mts * 8 + blockIdx.x % 8;
  if (cs >= cols * p.splits) return;
  const int t0 = q % mts * BM, col = cs % cols, split = cs / cols;
  const bool of_a = col >= n / kPartCols;
  const int g0 = (col - n / kPartCols) * 4;            // of A: its first group of 16 ranks
  int groups = 0;
  if (of_a) {
    int own[(BM + 63) / 64];
    uint64_t left[(BM + 63) / 64];
#pragma unroll
    for (int i = 0; i < (BM + 63) / 64; ++i) {
      const int r = i * 64 + lane;
      own[i] = r < BM && t0 + r < T ? a.adapter[t0 + r] : -1;
      if ((uint32_t)own[i] >= (uint32_t)a.sh.N) own[i] = -1;
      left[i] = __ballot(own[i] >= 0);
      if (r < BM) ids[r] = own[i];                     // every wave the same values
    }
    int count = 0;
#pragma unroll
    for (int i = 0; i < (BM + 63) / 64; ++i)
      for (; left[i]; ++count) {
        const int one = __builtin_amdgcn_readlane(own[i], __ffsll((unsigned long long)left[i]) - 1);
#pragma unroll
        for (int j = 0; j < (BM + 63) / 64; ++j) left[j] &= ~__ballot(own[j] == one);
        list[count] = one;
      }
    groups = count * per;
    if (g0 >= groups) return;
    __syncthreads();
  }

  // Loads: instruction i of a wave fills rows (4 i + wave) kPer + lane / kPieces, of one group of
  // 16 ranks where they are A's.
  const uint32_t row_bytes = (uint32_t)d * 2u;
  auto row_of = [&](int i) { return (i * 4 + wave) * kPer + lane / kPieces; };
  auto piece_of = [&](int row) { return (uint32_t)((lane % kPieces) ^ (RB == 256 ? row & 15 : (row >> 1) & 7)) << 4; };
  uint32_t x_off[kAI], w_off[kWI];
  const uint8_t* w_base[kWI];
#pragma unroll
  for (int i = 0; i < kAI; ++i) x_off[i] = (uint32_t)min(t0 + row_of(i), T - 1) * row_bytes + piece_of(row_of(i));
#pragma unroll
  for (int i = 0; i < kWI; ++i) {
    const int row = row_of(i);
    if (of_a) {
      const int g = min(g0 + (i * 4 + wave) * kPer / 16, groups - 1);
      const int id = __builtin_amdgcn_readfirstlane(list[g / per]);
      w_base[i] = reinterpret_cast<const uint8_t*>(a.a) + (size_t)id * rank * row_bytes;
      w_off[i] = (uint32_t)min(g % per * 16 + row % 16, rank - 1) * row_bytes + piece_of(row);
    } else {
      w_base[i] = reinterpret_cast<const uint8_t*>(a.w) + (size_t)col * kPartCols * row_bytes;
      w_off[i] = (uint32_t)row * row_bytes + piece_of(row);
    }
  }
  const int nk = d / (RB / 2), k0 = (int)((long)split * nk / p.splits), k1 = (int)((long)(split + 1) * nk / p.splits);
  auto load = [&](int step, int stage) {               // past the part's end: its last step, never read
    const size_t k = (size_t)min(step, k1 - 1) * RB;
    const uint32_t to = lds0 + stage * kStage;
#pragma unroll
    for (int i = 0; i < kWI; ++i) dma16(w_base[i] + k, w_off[i], to + kA + (i * 4 + wave) * 1024);
#pragma unroll
    for (int i = 0; i < kAI; ++i)
      dma16(reinterpret_cast<const uint8_t*>(a.x) + k, x_off[i], to + (i * 4 + wave) * 1024);
  };
#pragma unroll
  for (int s = 0; s < ST - 1; ++s) load(k0 + s, s);
  f32x4 acc[kN][kM] = {};
  const uint32_t swz = RB == 256 ? fr : (fr >> 1) & 7;
  int stage = 0;
  for (int step = k0; step < k1; ++step) {
    __builtin_amdgcn_s_waitcnt(wait_vm_lgkm0((ST - 2) * L));
    __syncthreads();                                   // the step has landed, the one before is read
    load(step + ST - 1, stage == 0 ? ST - 1 : stage - 1);
    const uint8_t* at = lds + stage * kStage;
#pragma unroll
    for (int s = 0; s < RB / 64; ++s) {
      u32x4 xf[kM], wf[kN];
      const uint32_t piece = ((4 * s + fc) ^ swz) << 4;
#pragma unroll
      for (int m = 0; m < kM; ++m) xf[m] = ld16(at + (wm * (BM / WM) + m * 16 + fr) * RB + piece);
#pragma unroll
      for (int j = 0; j < kN; ++j) wf[j] = ld16(at + kA + (wn * kN * 16 + j * 16 + fr) * RB + piece);
#pragma unroll
      for (int j = 0; j < kN; ++j)
#pragma unroll
        for (int m = 0; m < kM; ++m) acc[j][m] = mfma_bf16(wf[j], xf[m], acc[j][m]);
    }
    stage = stage == ST - 1 ? 0 : stage + 1;
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");     // no load outlives its LDS
  // A lane has columns 4 fc .. + 3 of token fr.
#pragma unroll
  for (int j = 0; j < kN; ++j)
#pragma unroll
    for (int m = 0; m < kM; ++m) {
      const int row = wm * (BM / WM) + m * 16 + fr, t = t0 + row, c = (wn * kN + j) * 16 + fc * 4;
      if (t >= T) continue;
      f32x4 v = acc[j][m];
      if (!of_a) {
        *reinterpret_cast<f32x4*>(p.part + ((size_t)split * T + t) * n + col * kPartCols + c) = v;
      } else {
        const int g = g0 + c / 16;
        if (g >= groups || ids[row] != list[g / per]) continue;
        const int r = g % per * 16 + c % 16;
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = r + i < rank ? v[i] : 0.f;
        *reinterpret_cast<f32x4*>(p.u + ((size_t)split * T + t) * pitch + r) = v;
      }
    }
}

// Parts of k added up in order, then bias, B u, activation: a block one token's 1024 columns, four
// a thread.
__global__ __launch_bounds__(256) void lora_finish_kernel(PartArgs p) {
  __shared__ __attribute__((aligned(16))) float su[kLoraMaxRank];
  const LoraArgs& a = p.a;
  const int T = a.sh.T, n = a.sh.n, rank = a.sh.rank, pitch = (rank + 15) / 16 * 16;
  const int t = blockIdx.x, c = (blockIdx.y * 256 + threadIdx.x) * 4;
  const int given = a.adapter[t], id = (uint32_t)given < (uint32_t)a.sh.N ? given : -1;
  const bool in = c < n;
  f32x4 v = {0.f, 0.f, 0.f, 0.f};
  u32x4 q[4][2] = {};
  const uint16_t* b = a.b + ((size_t)max(id, 0) * n + min(c, n - 4)) * rank;
  if (in && id >= 0) {                                 // the first 16 ranks, under way with the sums
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      q[i][0] = ld16(b + i * rank);
      if (rank > 8) q[i][1] = ld16(b + i * rank + 8);
    }
  }
  if (in) {
#pragma unroll 4
    for (int s = 0; s < p.splits; ++s) v += *reinterpret_cast<const f32x4*>(p.part + ((size_t)s * T + t) * n + c);
    if (a.bias) {
      const uint2 w = *reinterpret_cast<const uint2*>(a.bias + c);
      v[0] += __uint_as_float(w.x << 16);
      v[1] += __uint_as_float(w.x & 0xffff0000u);
      v[2] += __uint_as_float(w.y << 16);
      v[3] += __uint_as_float(w.y & 0xffff0000u);
    }
  }
  if (id >= 0) {
    if ((int)threadIdx.x < pitch) {
      float u = 0.f;
#pragma unroll 4
      for (int s = 0; s < p.splits; ++s) u += p.u[((size_t)s * T + t) * pitch + threadIdx.x];
      su[threadIdx.x] = u * (a.scale ? a.scale[id] : 1.f);
    }
    __syncthreads();
    if (in)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float s = dot8(q[i][0], su, 0.f);
        if (rank > 8) s = dot8(q[i][1], su + 8, s);
        for (int r = 16; r < rank; r += 8) s = dot8(ld16(b + i * rank + r), su + r, s);
        v[i] += s;
      }
  }
  if (!in) return;
  if (a.sh.f32_out) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = a.sh.gelu ? gelu_erf(v[i]) : v[i];
    *reinterpret_cast<f32x4*>(static_cast<float*>(a.y) + (size_t)t * n + c) = v;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = a.sh.gelu ? gelu_for_bf16(v[i]) : v[i];
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.y) + (size_t)t * n + c) =
        make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
  }
}

// ---- launches ------------------------------------------------------------------------------
enum LoraPath { kToken, kPart, kTile };

static LoraPath path_of(const LoraShape& s) {
  if (s.T == 1 && s.rank <= 32) return kToken;
  // Tiles need four steps of 64 k: their loads run two ahead, into the next tile only.
  return s.T > 512 && s.d >= 256 ? kTile : kPart;
}

// Tokens of a block, and the parts that k is cut into so that every CU has a block.
static int part_rows(const LoraShape& s) { return s.T <= 32 ? 32 : s.T <= 64 ? 64 : 128; }
static int part_splits(const LoraShape& s) {
  const int bm = part_rows(s), steps = s.d / (bm == 32 ? 128 : 64);
  const long tiles = (long)((s.T + bm - 1) / bm) * (s.n / kPartCols);
  return (int)std::max(1L, std::min({(256 + tiles / 2) / tiles, (long)steps / 2, 16L}));
}

size_t lora_u_bytes(const LoraShape& s) {
  const size_t T = s.T, pitch = lora_pitch(s.rank);
  switch (path_of(s)) {
    case kToken: return 256;
    case kTile: return T * pitch * 2 * lora_terms(s);
    default: return part_splits(s) * T * (s.n + pitch) * 4;
  }
}

template <int MT>
static void run_shrink(const LoraArgs& a, hipStream_t s) {
  lora_shrink_kernel<MT, 4, kWaves><<<(a.sh.T + 16 * MT - 1) / (16 * MT), kWaves * 64, 0, s>>>(a);
}

static hipError_t launch_part(const LoraArgs& a, hipStream_t s) {
  const LoraShape& h = a.sh;
  PartArgs p{a, part_splits(h), 0, static_cast<float*>(a.u), nullptr};
  p.u = p.part + (size_t)p.splits * h.T * h.n;
  const int bm = part_rows(h), mts = (h.T + bm - 1) / bm;
  p.a_tiles = (std::min(h.N, std::min(h.T, bm)) * (lora_pitch(h.rank) / 16) + 3) / 4;
  const int cs = (h.n / kPartCols + p.a_tiles) * p.splits;
  const unsigned grid = (unsigned)((cs + 7) / 8 * mts * 8);
  if (bm == 32) lora_part_kernel<32, 256, 3, 1><<<grid, 256, 0, s>>>(p);
  else if (bm == 64) lora_part_kernel<64, 128, 4, 2><<<grid, 256, 0, s>>>(p);
  else lora_part_kernel<128, 128, 3, 2><<<grid, 256, 0, s>>>(p);
  if (hipError_t e = hipGetLastError()) return e;
  lora_finish_kernel<<<dim3(h.T, (h.n + 1023) / 1024), 256, 0, s>>>(p);
  return hipGetLastError();
}

template <int RANKS>
static void launch_token(const LoraArgs& a, hipStream_t s) {
  const int n = a.sh.n;
  if (n >= 12288) lora_token_kernel<4, RANKS><<<(n + 63) / 64, kWaves * 64, 0, s>>>(a);
  else if (n >= 8192) lora_token_kernel<2, RANKS><<<(n + 31) / 32, kWaves * 64, 0, s>>>(a);
  else lora_token_kernel<1, RANKS><<<(n + 15) / 16, kWaves * 64, 0, s>>>(a);
}

hipError_t launch_lora(const LoraArgs& a, hipStream_t s) {
  switch (path_of(a.sh)) {
    case kToken:
      if (a.sh.rank <= 16) launch_token<1>(a, s);
      else launch_token<2>(a, s);
      return hipGetLastError();
    case kTile:
      if (a.sh.T > 16384) run_shrink<4>(a, s);
      else if (a.sh.T > 4096) run_shrink<2>(a, s);
      else run_shrink<1>(a, s);
      if (hipError_t e = hipGetLastError()) return e;
      return launch_lora_tile(a, s);
    default:
      return launch_part(a, s);
  }
}

}  // namespace moe
