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
#include "lora_parts.h"

namespace moe {

// ---------------------------------------------------------------------------
// u = scale A x before the tiled product, as bf16 terms.  A block has 32 tokens and first lists the
// different adapters among them; a few blocks share one tile's.  An adapter is pitch / 16 groups of 16
// ranks; a pass over k takes one, two or four groups, of one adapter or of several, so that x is
// read once for a few adapters.  x and A go into LDS in runs of 256 bytes of every row, as many
// stages as fit, pieces at piece ^ (row % 16); of a stage's 128 k each of the four waves multiplies
// 32, and their sums meet in LDS.  Bound by reading x: 16384 x 4096, 16 adapters of 16 ranks, 40 us, 3.4 TB/s; 8192 x 2816 of
// 32 ranks 13 us with one adapter, 19 with 64 requests of eight.
// ---------------------------------------------------------------------------
__global__ __launch_bounds__(256, 2) void lora_shrink_kernel(LoraArgs a) {
  constexpr int kRows = 32, kA = kRows * 256, LDS = 72 * 1024;   // two blocks a CU
  __shared__ __attribute__((aligned(1024))) uint8_t lds[LDS];
  __shared__ int list[kRows], ids[kRows];
  const int T = a.sh.T, d = a.sh.d, rank = a.sh.rank, pitch = lora_pitch(rank), per = pitch / 16;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int fr = lane & 15, fc = lane >> 4, t0 = blockIdx.x * kRows;
  const uint32_t lds0 = (uint32_t)(uintptr_t)lds, row_bytes = (uint32_t)d * 2u;
  if (threadIdx.x < kRows) ids[lane] = t0 + lane < T ? a.adapter[t0 + lane] : -1;
  const int all = lora_list<kRows>(a, t0, list) * per, nk = d / 128;
  // The block's share of the groups, in pairs.
  const int share = ((all + 1) / 2 + gridDim.y - 1) / gridDim.y * 2, from = blockIdx.y * share;
  const int groups = min(from + share, all);
  if (from >= all) return;
  __syncthreads();
  // Load i of a wave: four rows, of x first, then of A.
  auto row_of = [&](int i) { return (i * 4 + wave) * 4 + (lane >> 4); };

  // Groups g0 .. g0 + G - 1.
  auto pass = [&](auto g_tag, int g0) {
    constexpr int G = decltype(g_tag)::value, kRanks = 16 * G, kStage = (kRows + kRanks) * 256;
    constexpr int L = kStage / 4096, ST = LDS / kStage;          // 1 KB loads per wave and stage; stages
    static_assert(ST >= 3 && 4 * kRows * kRanks * 4 <= LDS && (ST - 2) * L < 64, "stages");
    const uint8_t* base[L];
    uint32_t off[L];
#pragma unroll
    for (int i = 0; i < L; ++i) {
      const int row = row_of(i), r = row - kRows;
      const uint32_t piece = (uint32_t)((lane & 15) ^ (row & 15)) << 4;
      if (i * 16 < kRows) {                            // 16 rows a load of all waves: of x or of A
        base[i] = reinterpret_cast<const uint8_t*>(a.x);
        off[i] = (uint32_t)min(t0 + row, T - 1) * row_bytes + piece;
      } else {
        const int g = min(g0 + (i * 16 - kRows) / 16, groups - 1);
        const int id = __builtin_amdgcn_readfirstlane(list[g / per]);
        base[i] = reinterpret_cast<const uint8_t*>(a.a) + (size_t)id * rank * row_bytes;
        off[i] = (uint32_t)min(g % per * 16 + r % 16, rank - 1) * row_bytes + piece;
      }
    }
    auto load = [&](int step, int stage) {             // past the end: the last step, never read
      const size_t k = (size_t)min(step, nk - 1) * 256;
#pragma unroll
      for (int i = 0; i < L; ++i) dma16(base[i] + k, off[i], lds0 + stage * kStage + (i * 4 + wave) * 1024);
    };
#pragma unroll
    for (int s = 0; s < ST - 1; ++s) load(s, s);
    f32x4 acc[G][2] = {};
    int stage = 0;
    for (int step = 0; step < nk; ++step) {
      __builtin_amdgcn_s_waitcnt(wait_vm_lgkm0((ST - 2) * L));
      __syncthreads();                                 // the step has landed, the one before is read
      load(step + ST - 1, stage == 0 ? ST - 1 : stage - 1);
      const uint8_t* at = lds + stage * kStage + (((4 * wave + fc) ^ fr) << 4);
      u32x4 xf[2], af[G];
#pragma unroll
      for (int m = 0; m < 2; ++m) xf[m] = ld16(at + (m * 16 + fr) * 256);
#pragma unroll
      for (int j = 0; j < G; ++j) af[j] = ld16(at + kA + (j * 16 + fr) * 256);
#pragma unroll
      for (int j = 0; j < G; ++j)
#pragma unroll
        for (int m = 0; m < 2; ++m) acc[j][m] = mfma_bf16(af[j], xf[m], acc[j][m]);
      stage = stage == ST - 1 ? 0 : stage + 1;
    }
    __builtin_amdgcn_s_waitcnt(wait_vm_lgkm0(0));      // no load lands any more
    __syncthreads();
    // The waves' sums by LDS: [wave][token][rank].  A lane has ranks 4 fc .. + 3 of token fr.
    float* part = reinterpret_cast<float*>(lds);
#pragma unroll
    for (int j = 0; j < G; ++j)
#pragma unroll
      for (int m = 0; m < 2; ++m)
        *reinterpret_cast<f32x4*>(part + ((wave * kRows + m * 16 + fr) * kRanks + j * 16 + fc * 4)) = acc[j][m];
    __syncthreads();
    for (int o = threadIdx.x; o < kRows * kRanks / 2; o += 256) {        // two ranks a thread
      const int row = o / (kRanks / 2), r = o % (kRanks / 2) * 2, g = g0 + r / 16, t = t0 + row;
      if (t >= T || g >= groups) continue;
      const int id = list[g / per], at_rank = g % per * 16 + r % 16;
      if (ids[row] != id) continue;
      float v[2] = {0.f, 0.f};
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        v[0] += part[(w * kRows + row) * kRanks + r];
        v[1] += part[(w * kRows + row) * kRanks + r + 1];
      }
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
  };
  for (int g0 = from; g0 < groups;) {
    if (groups - g0 == 1) {
      pass(std::integral_constant<int, 1>(), g0);
      ++g0;
    } else if (groups - g0 == 2) {
      pass(std::integral_constant<int, 2>(), g0);
      g0 += 2;
    } else {
      pass(std::integral_constant<int, 4>(), g0);
      g0 += 4;
    }
  }
}

// Eight values of B times eight of u, added to s.
__device__ __forceinline__ float dot8(const u32x4& q, const float* u, float s) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    s = fmaf(__uint_as_float(q[i] << 16), u[2 * i], s);
    s = fmaf(__uint_as_float(q[i] & 0xffff0000u), u[2 * i + 1], s);
  }
  return s;
}

// ---------------------------------------------------------------------------
// One token, bound by the bytes of W and by latency.  Every block works out u itself (A is read from
// memory once and then from L2), so one launch does all.  A wave takes whole rows, first of W, then
// its eighth of A's, in runs of 1 KB, P runs a set, three sets under way; x lies in LDS.  Lane j keeps
// the sum of the wave's j-th row of W and finishes it once u is there.  Products by the 4x4x4 MFMA: it
// multiplies four values of every lane of four with four of each of them, and the lane's own
// with its own is the one that is kept (16 cycles for 8 values; converting and multiplying
// them takes 96).  4096 x 4096, rank 16: 12.6 us, 2.7 TB/s; A and the end are 2.5 of them.  4096 -> 14336: 27
// us, 4.4 TB/s.
// ---------------------------------------------------------------------------
typedef short i16x4 __attribute__((ext_vector_type(4)));
// Lane l's four values (two words) of each operand: column l % 4 of the result's 4x4 block l / 4,
// of which row l % 4 is the lane's own times its own.
__device__ __forceinline__ f32x4 mfma_4x4(uint32_t a0, uint32_t a1, uint32_t b0, uint32_t b1, f32x4 c) {
  typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
  return __builtin_amdgcn_mfma_f32_4x4x4bf16_1k(__builtin_bit_cast(i16x4, (u32x2){a0, a1}),
                                                __builtin_bit_cast(i16x4, (u32x2){b0, b1}), c, 0, 0, 0);
}

// A block reads all of the adapter's A, so that is bounded (see path_of), and with it the width.
constexpr int kTokenWaves = 8, kTokenMostA = 128 * 1024, kTokenMaxWidth = kTokenMostA / 8;

template <int P>
__global__ __launch_bounds__(kTokenWaves * 64, 2) void lora_token_kernel(LoraArgs a) {
  constexpr int kSets = 3;
  __shared__ __attribute__((aligned(16))) uint16_t sx[kTokenMaxWidth];
  __shared__ __attribute__((aligned(16))) float su[kLoraMaxRank];
  const int d = a.sh.d, n = a.sh.n, rank = a.sh.rank;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int first = blockIdx.x * kTokenWaves + wave, stride = gridDim.x * kTokenWaves;   // rows of W
  const int segs = (d + P * 512 - 1) / (P * 512);
  const int of_w = first < n ? ((n - 1 - first) / stride + 1) * segs : 0;   // sets of W's rows
  const int total = of_w + rank / kTokenWaves * segs;  // and of A's (rank is a multiple of 8)
  const int turn = (wave + blockIdx.x / 8) % kTokenWaves;   // blocks of an XCD read different rows of A at a time
  const int given = a.adapter[0], id = (uint32_t)given < (uint32_t)a.sh.N ? given : -1;
  const int any = max(id, 0);                          // without an adapter A and B are read, not used
  const uint16_t* rows_a = a.a + ((size_t)any * rank + turn) * d;
  u32x4 v[kSets][P];
  // Set i: lane l has values 512 q + 8 l .. + 7 of its runs q; past the row's end any of its values.
  // Past the last set that one again, not used.
  auto load = [&](int slot, int i) {
    i = min(i, total - 1);
    const bool w = i < of_w;
    const int j = w ? i : i - of_w, s = j % segs;
    const uint16_t* p = w ? a.w + (size_t)(first + j / segs * stride) * d : rows_a + (size_t)(j / segs) * kTokenWaves * d;
#pragma unroll
    for (int q = 0; q < P; ++q) v[slot][q] = ld16(p + min((s * P + q) * 512 + lane * 8, d - 8));
  };
#pragma unroll
  for (int q = 0; q < kSets; ++q) load(q, q);
  for (int i = threadIdx.x * 8; i < d; i += kTokenWaves * 64 * 8) st16(sx + i, ld16(a.x + i));
  // The lane's own row: 16 ranks of its B, its bias; and the scale.
  const int row = min(first + lane * stride, n - 1);
  const uint16_t* b = a.b + ((size_t)any * n + row) * rank;
  const u32x4 b0 = ld16(b), b1 = rank > 8 ? ld16(b + 8) : u32x4{0, 0, 0, 0};
  const float bias = a.bias ? bf16_to_f32(a.bias[row]) : 0.f, scale = a.scale ? a.scale[any] : 1.f;
  __syncthreads();
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  float mine = 0.f;
  auto use = [&](int slot, int i) {
    const bool w = i < of_w;
    const int j = w ? i : i - of_w, s = j % segs;
#pragma unroll
    for (int q = 0; q < P; ++q) {
      const int k = (s * P + q) * 512 + lane * 8;
      const u32x4 zero = {0, 0, 0, 0}, x = k < d ? ld16(sx + min(k, d - 8)) : zero, y = k < d ? v[slot][q] : zero;
      acc = mfma_4x4(y[0], y[1], x[0], x[1], acc);
      acc = mfma_4x4(y[2], y[3], x[2], x[3], acc);
    }
    if (s + 1 < segs) return;
    const int own = lane & 3;
    const float sum = wave_sum_f(own == 0 ? acc[0] : own == 1 ? acc[1] : own == 2 ? acc[2] : acc[3]);
    if (w) mine = lane == j / segs ? sum : mine;
    else if (lane == 0) su[j / segs * kTokenWaves + turn] = sum * scale;
    acc = f32x4{0.f, 0.f, 0.f, 0.f};
  };
  for (int i = 0; i < total; i += kSets) {
#pragma unroll
    for (int q = 0; q < kSets; ++q) {
      if (i + q < total) use(q, i + q);
      load(q, i + q + kSets);
    }
  }
  __syncthreads();
  if (first + lane * stride >= n) return;
  float sum = mine + bias;
  if (id >= 0) {
    float s = dot8(b0, su, 0.f);
    if (rank > 8) s = dot8(b1, su + 8, s);
    for (int r = 16; r < rank; r += 8) s = dot8(ld16(b + r), su + r, s);
    sum += s;
  }
  if (a.sh.f32_out) static_cast<float*>(a.y)[row] = a.sh.gelu ? gelu_f32(sum) : sum;
  else static_cast<uint16_t*>(a.y)[row] = (uint16_t)pack_bf16x2(a.sh.gelu ? gelu_for_bf16(sum) : sum, 0.f);
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
// the other's loads.  32 tokens, 4096 -> 14336, 32 adapters: 24 to 27 us, 4.9 TB/s at best, then the second
// kernel's 5.5.
// ---------------------------------------------------------------------------
constexpr int kPartCols = 64;

template <int BM, int RB, int ST, int WM, int OCC>
__global__ __launch_bounds__(256, OCC) void lora_part_kernel(LoraPartArgs p) {
  constexpr int kPieces = RB / 16, kPer = 1024 / RB;             // of a row; rows per load
  constexpr int kA = BM * RB, kStage = (BM + kPartCols) * RB;
  constexpr int kAI = kA / 4096, kWI = kPartCols * RB / 4096, L = kAI + kWI;   // loads per wave
  constexpr int kM = BM / WM / 16, kN = kPartCols * WM / 64;     // 16x16 tiles per wave
  static_assert(kA % 4096 == 0 && OCC * (ST * kStage + BM * 4) <= 160 * 1024 && (ST - 2) * L < 64, "LDS plan");
  __shared__ __attribute__((aligned(1024))) uint8_t lds[ST * kStage];
  __shared__ int list[BM];
  const LoraArgs& a = p.a;
  const int T = a.sh.T, d = a.sh.d, n = a.sh.n, rank = a.sh.rank, pitch = lora_pitch(rank), per = pitch / 16;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int fr = lane & 15, fc = lane >> 4, wm = wave % WM, wn = wave / WM;
  const uint32_t lds0 = (uint32_t)(uintptr_t)lds;
  LoraUnit w;
  if (!lora_unit<BM, kPartCols>(p, w)) return;
  int groups = 0;
  if (w.of_a) {
    groups = lora_list<BM>(a, w.t0, list) * per;
    if (w.g0 >= groups) return;
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
  for (int i = 0; i < kAI; ++i) x_off[i] = (uint32_t)min(w.t0 + row_of(i), T - 1) * row_bytes + piece_of(row_of(i));
#pragma unroll
  for (int i = 0; i < kWI; ++i) {
    const int row = row_of(i);
    if (w.of_a) {
      const int g = min(w.g0 + (i * 4 + wave) * kPer / 16, groups - 1);
      const int id = __builtin_amdgcn_readfirstlane(list[g / per]);
      w_base[i] = reinterpret_cast<const uint8_t*>(a.a) + (size_t)id * rank * row_bytes;
      w_off[i] = (uint32_t)min(g % per * 16 + row % 16, rank - 1) * row_bytes + piece_of(row);
    } else {
      w_base[i] = reinterpret_cast<const uint8_t*>(a.w) + (size_t)w.n0 * row_bytes;
      w_off[i] = (uint32_t)row * row_bytes + piece_of(row);
    }
  }
  // In steps of RB bytes; runs of 256 bytes start at whole ones, so the parts' borders are even.
  const int k0 = w.k0 * 128 / RB, k1 = w.split + 1 < p.splits ? w.k1 * 128 / RB : d * 2 / RB;
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
  for (int m = 0; m < kM; ++m) {
    const int t = w.t0 + wm * (BM / WM) + m * 16 + fr;
    if (t >= T) continue;
    const int id = w.of_a ? a.adapter[t] : -1;
#pragma unroll
    for (int j = 0; j < kN; ++j) {
      const int c = (wn * kN + j) * 16 + fc * 4;
      f32x4 v = acc[j][m];
      if (!w.of_a) {
        *reinterpret_cast<f32x4*>(p.part + ((size_t)w.split * T + t) * n + w.n0 + c) = v;
      } else {
        const int g = w.g0 + c / 16;
        if (g >= groups || id != list[g / per]) continue;
        const int r = g % per * 16 + c % 16;
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = r + i < rank ? v[i] : 0.f;
        *reinterpret_cast<f32x4*>(p.u + ((size_t)w.split * T + t) * pitch + r) = v;
      }
    }
  }
}

// Parts of k added up in order, then bias, B u, activation.  A block has 1024 columns of one token, a
// thread every 256th of them: B's columns lie side by side, so lanes that take neighbours read
// whole lines (four neighbours a thread read 64 lines of 128 bytes with every load: 16 us for 512 x 4096).
__global__ __launch_bounds__(256) void lora_finish_kernel(LoraPartArgs p) {
  constexpr int kCols = 4;
  __shared__ __attribute__((aligned(16))) float su[kLoraMaxRank];
  const LoraArgs& a = p.a;
  const int T = a.sh.T, n = a.sh.n, rank = a.sh.rank, pitch = lora_pitch(rank);
  const int t = blockIdx.x, c0 = blockIdx.y * 256 * kCols + threadIdx.x;
  float v[kCols];
#pragma unroll
  for (int i = 0; i < kCols; ++i) v[i] = p.part[(size_t)t * n + min(c0 + i * 256, n - 1)];
  const int given = a.adapter[t], id = (uint32_t)given < (uint32_t)a.sh.N ? given : -1;
  const uint16_t* b = a.b + (size_t)max(id, 0) * n * rank;
  u32x4 q[kCols][2] = {};
  if (id >= 0) {                                       // the first 16 ranks, under way with the sums
#pragma unroll
    for (int i = 0; i < kCols; ++i) {
      const uint16_t* row = b + (size_t)min(c0 + i * 256, n - 1) * rank;
      q[i][0] = ld16(row);
      if (rank > 8) q[i][1] = ld16(row + 8);
    }
  }
  for (int s = 1; s < p.splits; ++s)
#pragma unroll
    for (int i = 0; i < kCols; ++i) v[i] += p.part[((size_t)s * T + t) * n + min(c0 + i * 256, n - 1)];
  if (a.bias)
#pragma unroll
    for (int i = 0; i < kCols; ++i) v[i] += bf16_to_f32(a.bias[min(c0 + i * 256, n - 1)]);
  if (id >= 0) {
    if ((int)threadIdx.x < pitch) {
      float u = 0.f;
#pragma unroll 4
      for (int s = 0; s < p.splits; ++s) u += p.u[((size_t)s * T + t) * pitch + threadIdx.x];
      su[threadIdx.x] = u * (a.scale ? a.scale[id] : 1.f);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kCols; ++i) {
      const uint16_t* row = b + (size_t)min(c0 + i * 256, n - 1) * rank;
      float s = dot8(q[i][0], su, 0.f);
      if (rank > 8) s = dot8(q[i][1], su + 8, s);
      for (int r = 16; r < rank; r += 8) s = dot8(ld16(row + r), su + r, s);
      v[i] += s;
    }
  }
#pragma unroll
  for (int i = 0; i < kCols; ++i) {
    const int c = c0 + i * 256;
    if (c >= n) continue;
    if (a.sh.f32_out) static_cast<float*>(a.y)[(size_t)t * n + c] = a.sh.gelu ? gelu_f32(v[i]) : v[i];
    else static_cast<uint16_t*>(a.y)[(size_t)t * n + c] = (uint16_t)pack_bf16x2(a.sh.gelu ? gelu_for_bf16(v[i]) : v[i], 0.f);
  }
}

// ---- launches ------------------------------------------------------------------------------
enum LoraPath { kToken, kPart, kTile };

// Tokens of a part's block, and the parts that k is cut into, so that every CU has a block, or
// nearly two where k is long.  96 to 512 tokens, n = 4096: d = 4096 in 256 blocks 25 to 50 us, in 448 26
// to 52; d = 14336 50 to 125 and 43 to 116.
static int part_rows(const LoraShape& s) { return s.T <= 32 ? 32 : s.T <= 64 ? 64 : 128; }
static long part_tiles(const LoraShape& s) {
  const int bm = part_rows(s), bn = bm == 128 ? 128 : kPartCols;
  return (long)((s.T + bm - 1) / bm) * ((s.n + bn - 1) / bn);
}
static int part_splits(const LoraShape& s) {
  const long tiles = part_tiles(s), want = tiles <= 128 && s.d >= 8192 ? 448 : 256;
  // at least 128 k each, and whole runs of 256 bytes
  return (int)std::max(1L, std::min({(want + tiles / 2) / tiles, (long)s.d / 128, 16L}));
}

static LoraPath path_of(const LoraShape& s) {
  // One token, us by this way (A's values) and in parts: n = d = 4096, 64 K 14 and 16, 256 K 20 and 20;
  // 14336 x 4096, 224 K 33 and 34, 448 K 39 and 36; 2048 x 2816, 64 K 9 and 12.
  if (s.T == 1 && (long)s.rank * s.d <= kTokenMostA && s.n <= 64 * 256 * kTokenWaves)   // a lane for a wave's every row
    return kToken;
  // Tiles need four steps of 64 k: their loads run two ahead, into the next tile only.
  return s.T > 128 && s.d >= 256 && part_splits(s) == 1 ? kTile : kPart;
}

size_t lora_u_bytes(const LoraShape& s) {
  const size_t T = s.T, pitch = lora_pitch(s.rank);
  switch (path_of(s)) {
    case kToken: return 256;
    case kTile: return T * pitch * 2 * lora_terms(s);
    default: return part_splits(s) * T * (s.n + pitch) * 4;
  }
}

// Blocks that share a tile's groups: those without any end at once.  8192 x 2816, 64 requests of 8 adapters of
// 32 ranks: two a tile 22 us, four 19; scattered adapters gain by eight where tiles are few.
static void launch_shrink(const LoraArgs& a, hipStream_t s) {
  const int tiles = (a.sh.T + 31) / 32;
  lora_shrink_kernel<<<dim3(tiles, tiles <= 128 ? 8 : 4), 256, 0, s>>>(a);
}

static hipError_t launch_part(const LoraArgs& a, hipStream_t s) {
  const LoraShape& h = a.sh;
  LoraPartArgs p{a, part_splits(h), 0, static_cast<float*>(a.u), nullptr};
  p.u = p.part + (size_t)p.splits * h.T * h.n;
  const int bm = part_rows(h), bn = bm == 128 ? 128 : kPartCols, mts = (h.T + bm - 1) / bm;
  p.a_tiles = (std::min(h.N, std::min(h.T, bm)) * (lora_pitch(h.rank) / 16) * 16 + bn - 1) / bn;
  const int cs = ((h.n + bn - 1) / bn + p.a_tiles) * p.splits;
  const unsigned grid = (unsigned)((cs + 7) / 8 * mts * 8);
  if (bm == 32) lora_part_kernel<32, 256, 3, 1, 2><<<grid, 256, 0, s>>>(p);
  else if (bm == 64) lora_part_kernel<64, 128, 4, 2, 2><<<grid, 256, 0, s>>>(p);
  else launch_lora_part_tile(p, grid, s);
  if (hipError_t e = hipGetLastError()) return e;
  lora_finish_kernel<<<dim3(h.T, (h.n + 1023) / 1024), 256, 0, s>>>(p);
  return hipGetLastError();
}

static void launch_token(const LoraArgs& a, hipStream_t s) {
  const int blocks = std::min(256, (a.sh.n + kTokenWaves - 1) / kTokenWaves);
  if (a.sh.d <= 1024) lora_token_kernel<2><<<blocks, kTokenWaves * 64, 0, s>>>(a);
  else if (a.sh.d <= 2048) lora_token_kernel<4><<<blocks, kTokenWaves * 64, 0, s>>>(a);
  else lora_token_kernel<8><<<blocks, kTokenWaves * 64, 0, s>>>(a);
}

hipError_t launch_lora(const LoraArgs& a, hipStream_t s) {
  switch (path_of(a.sh)) {
    case kToken:
      launch_token(a, s);
      return hipGetLastError();
    case kTile:
      launch_shrink(a, s);
      if (hipError_t e = hipGetLastError()) return e;
      return launch_lora_tile(a, s);
    default:
      return launch_part(a, s);
  }
}

}  // namespace moe
