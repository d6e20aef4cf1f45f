// Grouped expert products with MXFP4 weights on gfx950.
//
// out[r] = a[r] W_e^T + b_e for the rows of expert e's segment, W_e [N][K] as e2m1 codes
// with one e8m0 scale per 32 values of k; the first product applies the exact-erf GELU.
#include <algorithm>
#include <type_traits>

#include "device_common.h"
#include "mx.h"
#include "mx_tiles.h"

namespace moe {

// ---------------------------------------------------------------------------
// Weight streaming (few rows per expert: bound by the bytes of the codes).
//
// Tile = 16 NMT rows of one expert x 128 output columns, 8 waves of 16 columns; persistent
// blocks, one per CU.  k goes in runs of RUN values through S LDS stages filled by DMA:
// whole 128 B or 256 B runs of each code row, whole runs of the activations, 16 bytes of
// each row's scales.  (Codes loaded straight to registers in the MFMA's layout, 64 B of 16
// rows at a time, streamed at 3.2 TB/s whatever the rest of the kernel did.)  The loads run
// S - 1 runs ahead and on into the block's next tile.
// Codes are widened to bf16 by v_cvt_scalef32_pk_bf16_fp4 (exact, scale included) and
// multiplied by MFMA 16x16x32 with W as the first operand; slice s of a 128-k granule takes k =
// 32 q + 8 s .. + 7 of lane group q from both operands, so a lane's 16 bytes of codes are one
// scale block and four slices.
// LDS: 16 B pieces of an activation row at piece ^ (row % 16) within each 256 B, of a code row
// at piece ^ (row % 16) (256 B rows) or piece ^ ((row >> 1) & 7) (128 B rows): 16 rows' reads
// of one piece touch every bank once.
// With `splits` > 1 a tile is one part of k, summed into `partial`.
// 32 tokens x 2 of 8 experts, d = 4096, F = 14336, weights from memory: up 53 us, down 48 to 53
// by the box, 4.7 to 5.2 TB/s of codes and scales, a copy's 4.8 read and written.  Down has 32
// column tiles, 256 in all while no expert has more than 16 rows; one that has makes a second
// round, 70 us.  (Up's last round has half the blocks; giving those tiles to all blocks
// by halves measured the same: the bytes take their time either way.)
// ---------------------------------------------------------------------------
constexpr int kStreamWaves = 8, kStreamCols = kStreamWaves * 16, kStreamBlocks = 256;

struct StreamArgs {
  const uint16_t* a;       // [rows of a][K]
  const int32_t* src;      // or null
  int k_top, tokens;
  const int32_t* offsets;
  int E, rows, N, K;
  const uint8_t* w;
  const uint8_t* ws;
  const uint16_t* bias;
  void* out;
  int splits;
  float* partial;
};

// Words at the same address for all lanes, through the scalar cache: a vector load would be
// waited for behind every load to LDS in flight.
typedef __attribute__((address_space(4))) const uint32_t scalar_u32;
__device__ __forceinline__ scalar_u32* scalar_words(const void* p) {
  return (scalar_u32*)reinterpret_cast<uintptr_t>(p);
}

template <bool UP, int NMT, int RUN, int S>
__global__ __launch_bounds__(512, 1) void mx_stream_kernel(StreamArgs p) {
  constexpr int kRows = 16 * NMT, G = RUN / 128;               // granules per run
  constexpr int kARow = RUN * 2, kWRow = RUN / 2;              // bytes per row and run
  constexpr int kA = kRows * kARow, kW = kStreamCols * kWRow, kS = kStreamCols * 16;
  constexpr int kStage = kA + kW + kS, oW = kA, oS = kA + kW;
  constexpr int kAI = kA / 8192, kWI = kW / 8192, L = kAI + kWI;   // 1 KB loads per wave
  constexpr int kALanes = kARow / 16, kWLanes = kWRow / 16;    // lanes per row (A: at most 64)
  static_assert(kA % 8192 == 0 && kW % 8192 == 0 && (kALanes == 64 || kALanes == 32), "load plan");
  static_assert(S * kStage + sizeof(TileTable) <= 160 * 1024, "LDS");
  __shared__ __attribute__((aligned(1024))) uint8_t lds[S * kStage];
  __shared__ TileTable table;

  const int N = p.N, K = p.K, lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int fr = lane & 15, fc = lane >> 4;
  const uint32_t lds0 = (uint32_t)(uintptr_t)lds;
  const int granules = K / 128, ntn = (N + kStreamCols - 1) / kStreamCols;
  const uint32_t w_pitch = K / 2, s_pitch = K / 32;
  const int mts = fill_tiles<kRows>(p.offsets, p.E, p.rows, table);
  const int units = mts * ntn * p.splits;        // rows * N is under 2^31

  // A unit of work: a tile and a part of its k; row tiles of one column tile are neighbours.
  struct Unit {
    int e, r0, r1, n0, split, g0, runs, g1;
  };
  auto locate = [&](int u, Unit& w) {
    if (u >= units) return false;
    const int mt = u % mts, rest = u / mts;
    w.split = rest % p.splits;
    w.n0 = rest / p.splits * kStreamCols;
    w.g0 = (int)((long)w.split * granules / p.splits);
    w.g1 = (int)((long)(w.split + 1) * granules / p.splits);
    w.runs = (w.g1 - w.g0 + G - 1) / G;
    return find_tile<kRows>(table, mt, w.e, w.r0, w.r1);
  };

  // ---- loads ----
  uint32_t a_off[kAI], a_max[kAI];                 // bytes; the row's last 16
  uint32_t w_off, s_off;
  const uint8_t *w_base, *s_base;
  uint32_t w_last;                                 // of the expert's codes: its last 16 bytes
  const int w_row = wave * (64 / kWLanes) + lane / kWLanes;   // load i: 8 waves' rows further on
  auto aim = [&](const Unit& w) {
#pragma unroll
    for (int i = 0; i < kAI; ++i) {
      constexpr int kPer = 64 / kALanes;           // rows per load: 1 or 2
      const int row = (i * 8 + wave) * kPer + lane / kALanes;
      uint32_t tok = (uint32_t)min(w.r0 + row, w.r1 - 1);
      if (p.src) {
        const int r = min(w.r0 + (i * 8 + wave) * kPer, w.r1 - 1);
        tok = scalar_words(p.src)[r];
        if (kPer == 2) {
          const uint32_t second = scalar_words(p.src)[min(r + 1, w.r1 - 1)];
          tok = lane / kALanes ? second : tok;
        }
        tok = min(tok / (uint32_t)p.k_top, (uint32_t)p.tokens - 1u);
      }
      a_off[i] = tok * (uint32_t)K * 2u + ((lane % kALanes) ^ (row & 15)) * 16u + (uint32_t)w.g0 * 256u;
      a_max[i] = tok * (uint32_t)K * 2u + (uint32_t)K * 2u - 16u;
    }
    const size_t first = (size_t)w.e * N;
    w_base = p.w + first * w_pitch;
    w_last = (uint32_t)N * w_pitch - 16u;
    s_base = p.ws + first * s_pitch;
    // Columns past N read the last one.  A run past the row's end reads the next row's
    // codes and scales (never used), past the expert's last byte its last ones.
    w_off = (uint32_t)w.g0 * 64u;
    s_off = (uint32_t)min(w.n0 + (wave & 1) * 64 + lane, N - 1) * s_pitch + (uint32_t)w.g0 * 4u;
  };
  // The loads have a unit of their own, any number ahead of the one being multiplied.
  Unit cur, next;
  int u = blockIdx.x, u_load = blockIdx.x;
  if (!locate(u, cur)) return;
  next = cur;
  bool more = true;
  aim(cur);
  int ls = 0;                                      // run to load next
  const uint32_t s_last = (uint32_t)N * s_pitch - 16u;
  auto load = [&](int i, int stage) {
    const uint32_t base = lds0 + stage * kStage;
    if (i < kAI) {
      dma16(p.a, min(a_off[i < kAI ? i : 0] + (uint32_t)ls * kARow, a_max[i < kAI ? i : 0]),
            base + (i * 8 + wave) * 1024);
    } else {
      const int row = (i - kAI) * (512 / kWLanes) + w_row;
      const int c = (lane % kWLanes) ^ (kWLanes == 16 ? row & 15 : (row >> 1) & 7);
      const uint32_t at = (uint32_t)min(next.n0 + row, N - 1) * w_pitch + w_off + (uint32_t)ls * kWRow + c * 16;
      dma16(w_base, min(at, w_last), base + oW + ((i - kAI) * 8 + wave) * 1024);
    }
  };
  // The scales: two loads of 64 columns, by the first two waves.
  auto load_s = [&](int stage) {
    if (wave < 2) dma16(s_base, min(s_off + (uint32_t)ls * (G * 4), s_last), lds0 + stage * kStage + oS + wave * 1024);
  };
  auto advance = [&]() {
    if (++ls < next.runs) return;
    if (more) {
      u_load += gridDim.x;
      Unit w;
      more = locate(u_load, w);
      if (more) {
        next = w;
        aim(w);
        ls = 0;
        return;
      }
    }
    ls = next.runs - 1;                            // repeated into free stages, never read
  };
  auto landed = [&]() {                            // every load but the last S - 2 runs'
    if (wave < 2) __builtin_amdgcn_s_waitcnt(wait_vm((S - 2) * (L + 1)));
    else __builtin_amdgcn_s_waitcnt(wait_vm((S - 2) * L));
  };

  f32x4 acc[NMT];
  const uint32_t w_lane = oW + (wave * 16 + fr) * kWRow, swz = kWLanes == 16 ? fr : (fr >> 1) & 7;
  // One granule for MA active row tiles: every fragment read first, then the products.
  auto granule = [&](auto ma, const uint8_t* st, int i, uint32_t sw) {
    constexpr int MA = decltype(ma)::value;
    const u32x4 codes = ld16(st + w_lane + (((4 * i + fc) ^ swz) << 4));
    u32x4 af[4][MA];
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
      for (int m = 0; m < MA; ++m)
        af[s][m] = ld16(st + (m * 16 + fr) * kARow + i * 256 + (((4 * fc + s) ^ fr) << 4));
    const float scale = __uint_as_float(((sw >> (8 * fc)) & 0xffu) << 23);
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      u32x4 wf;
      wf[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes[s], scale, 0));
      wf[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes[s], scale, 1));
      wf[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes[s], scale, 2));
      wf[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes[s], scale, 3));
#pragma unroll
      for (int m = 0; m < MA; ++m) acc[m] = mfma_bf16(wf, af[s][m], acc[m]);
    }
  };

  // ---- S - 1 runs in flight, then run by run ----
#pragma unroll
  for (int s = 0; s < S - 1; ++s) {
#pragma unroll
    for (int i = 0; i < L; ++i) load(i, s);
    load_s(s);
    advance();
  }
  int st = 0;
  for (;;) {
#pragma unroll
    for (int m = 0; m < NMT; ++m) acc[m] = f32x4{0.f, 0.f, 0.f, 0.f};
    const int active = (cur.r1 - cur.r0 + 15) >> 4;
    // Where the row's scales lie in their 16 bytes (moved back only at the expert's last ones).
    const uint32_t s_want = (uint32_t)min(cur.n0 + wave * 16 + fr, N - 1) * s_pitch + (uint32_t)cur.g0 * 4u;
    auto run = [&](auto ma) {
      for (int c = 0; c < cur.runs; ++c) {
        landed();
        __syncthreads();                           // for all; the run before is read
        const uint8_t* base = lds + st * kStage;
        const int into = st == 0 ? S - 1 : st - 1;
        const uint32_t want = s_want + (uint32_t)c * (G * 4);
        const uint8_t* sp = base + oS + (wave * 16 + fr) * 16 + (want - min(want, s_last));
#pragma unroll
        for (int i = 0; i < G; ++i) {
          const uint32_t sw = *reinterpret_cast<const uint32_t*>(sp + i * 4);
          if (cur.g0 + c * G + i < cur.g1) granule(ma, base, i, sw);
#pragma unroll
          for (int j = i * L / G; j < (i + 1) * L / G; ++j) load(j, into);
          if (i == G - 1) load_s(into);
          __builtin_amdgcn_sched_barrier(0);
        }
        advance();
        st = st == S - 1 ? 0 : st + 1;
      }
    };
    if (NMT == 1 || active == 1) run(std::integral_constant<int, 1>{});
    else run(std::integral_constant<int, NMT>{});

    // Lane: row m*16 + fr, columns n0 + 16 wave + 4 fc .. + 3.
    const int n = cur.n0 + wave * 16 + 4 * fc;
    uint2 b = make_uint2(0u, 0u);
    if (p.bias && p.splits == 1) {                 // the wave's 16 columns
      scalar_u32* w = scalar_words(p.bias + (size_t)cur.e * N + min(cur.n0 + wave * 16, N - 16));
      const uint32_t q[8] = {w[0], w[1], w[2], w[3], w[4], w[5], w[6], w[7]};
      b = fc < 2 ? (fc == 0 ? make_uint2(q[0], q[1]) : make_uint2(q[2], q[3]))
                 : (fc == 2 ? make_uint2(q[4], q[5]) : make_uint2(q[6], q[7]));
    }
#pragma unroll
    for (int m = 0; m < NMT; ++m) {
      const int r = cur.r0 + m * 16 + fr;
      if (m >= active || r >= cur.r1 || n >= N) continue;
      f32x4 v = acc[m];
      if (p.splits > 1) {
        *reinterpret_cast<f32x4*>(p.partial + ((size_t)cur.split * p.rows + r) * N + n) = v;
        continue;
      }
      v[0] += __uint_as_float(b.x << 16);
      v[1] += __uint_as_float(b.x & 0xffff0000u);
      v[2] += __uint_as_float(b.y << 16);
      v[3] += __uint_as_float(b.y & 0xffff0000u);
      if constexpr (UP)
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + (size_t)r * N + n) =
            make_uint2(pack_bf16x2(gelu_for_bf16(v[0]), gelu_for_bf16(v[1])), pack_bf16x2(gelu_for_bf16(v[2]), gelu_for_bf16(v[3])));
      else
        *reinterpret_cast<f32x4*>(static_cast<float*>(p.out) + (size_t)r * N + n) = v;
    }
    u += gridDim.x;
    if (!locate(u, cur)) break;
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); // no load outlives its LDS
}

// The parts of k summed in order, then bias and GELU.  Block = rows blockIdx.y of the
// dispatch; its expert is found from the offsets.
template <bool UP>
__global__ __launch_bounds__(256) void mx_split_sum_kernel(
    const int32_t* __restrict__ offsets, int E, int rows_cap, const uint16_t* __restrict__ bias,
    void* __restrict__ out, int N, int splits, const float* __restrict__ partial) {
  const int r = blockIdx.y, n = (blockIdx.x * 256 + threadIdx.x) * 4;
  int e = 0;
  if (bias) {
    // The expert of row r: as many offsets [1, E] as are <= r lie before it.
    int before = 0;
    for (int i = threadIdx.x & 63; i < E; i += 64) before += offsets[i + 1] <= r;
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) before += __shfl_xor(before, o);
    e = min(before, E - 1);
  }
  if (n >= N || r < offsets[0] || r >= min(offsets[E], rows_cap)) return;
  f32x4 v = *reinterpret_cast<const f32x4*>(partial + (size_t)r * N + n);
  for (int s = 1; s < splits; ++s)
    v += *reinterpret_cast<const f32x4*>(partial + ((size_t)s * rows_cap + r) * N + n);
  if (bias) {
    const uint2 b = *reinterpret_cast<const uint2*>(bias + (size_t)e * N + n);
    v[0] += __uint_as_float(b.x << 16);
    v[1] += __uint_as_float(b.x & 0xffff0000u);
    v[2] += __uint_as_float(b.y << 16);
    v[3] += __uint_as_float(b.y & 0xffff0000u);
  }
  if constexpr (UP)
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(out) + (size_t)r * N + n) =
        make_uint2(pack_bf16x2(gelu_for_bf16(v[0]), gelu_for_bf16(v[1])), pack_bf16x2(gelu_for_bf16(v[2]), gelu_for_bf16(v[3])));
  else
    *reinterpret_cast<f32x4*>(static_cast<float*>(out) + (size_t)r * N + n) = v;
}

// Parts of k on the streaming path: enough units for every CU from the experts that can have
// rows, at least 512 of k in each part, and only while the partial sums stay small beside
// the codes (at most 64 rows in all).
static int stream_splits(int T, int k, int E, int N, int K) {
  const long rows = (long)T * k;
  if (rows > 64) return 1;
  const long tiles = std::min<long>(E, rows) * ((N + kStreamCols - 1) / kStreamCols);
  return (int)std::max(1L, std::min({8L, K / 512L, kStreamBlocks / tiles}));
}

size_t mx_partial_bytes(int T, int k, int E, int N, int K) {
  const int s = stream_splits(T, k, E, N, K);
  return s > 1 ? (size_t)s * T * k * N * 4 : 0;
}

// Experts averaging many rows run the LDS-tiled kernel, the rest stream: from 32 rows with
// fp4 activations, whose matrix products take a quarter of the time, from 56 with bf16 ones.
// Streamed and tiled, us: E = 8, K = 4096, N = 14336: fp4 24 rows 70 and 66, 36 rows 119 and
// 67; bf16 48 rows 115 and 119, 72 rows 179 and 120.  E = 64, K = 2048, N = 1408: fp4 24 rows 36
// and 39, 36 rows 54 and 40; bf16 48 rows 61 and 65, 72 rows 89 and 73.  The tiled kernel's loads
// run up to two steps of 256 k ahead, so it starts at k = 512.
static bool tiled(long rows, int E, int K, bool fp4) { return rows >= (fp4 ? 32L : 56L) * E && K >= 512; }

size_t mx_act_bytes(int T, int k, int E, int N, int K, bool fp4) {
  const long rows = (long)T * k;
  return tiled(rows, E, K, fp4) ? mx_tile_bytes(rows, E, N, K, fp4) : fp4 ? (size_t)rows * K * 2 : 0;
}

template <bool UP>
static void launch_stream(const MxFfnArgs& a, const void* act, hipStream_t s) {
  const int R = a.T * a.k, splits = stream_splits(a.T, a.k, a.E, a.N, a.K);
  StreamArgs p{};
  p.a = static_cast<const uint16_t*>(act);
  p.src = a.src;
  p.k_top = a.k;
  p.tokens = a.T;
  p.offsets = a.offsets;
  p.E = a.E;
  p.rows = R;
  p.N = a.N;
  p.K = a.K;
  p.w = a.w;
  p.ws = a.ws;
  p.bias = static_cast<const uint16_t*>(a.bias);
  p.out = a.out;
  p.splits = splits;
  p.partial = a.partial;
  // Tiles of 16 rows and runs of 512 while experts average at most 12, else 32 rows and runs
  // of 256 (the activations' share of the LDS): E = 8, K = 4096, N = 14336, 12 rows 45 and 50 us,
  // 18 rows 75 and 69; E = 64, K = 2048, N = 1408, 9 rows 22 and 24 us, 18 rows 33 and 32.
  if ((long)R <= 12L * a.E) mx_stream_kernel<UP, 1, 512, 3><<<kStreamBlocks, 512, 0, s>>>(p);
  else mx_stream_kernel<UP, 2, 256, 4><<<kStreamBlocks, 512, 0, s>>>(p);
  if (splits > 1)
    mx_split_sum_kernel<UP><<<dim3((a.N / 4 + 255) / 256, R), 256, 0, s>>>(
        a.offsets, a.E, R, p.bias, a.out, a.N, splits, a.partial);
}

hipError_t launch_mx_ffn(const MxFfnArgs& a, hipStream_t s) {
  if (tiled((long)a.T * a.k, a.E, a.K, a.fp4)) return launch_mx_tile(a, s);
  const void* act = a.a;
  if (a.fp4) {
    // The values the 4-bit activations stand for, as bf16: exact in the products.
    if (hipError_t e = launch_mx_requantize(a.a, a.a_rows, a.K, a.act, s)) return e;
    act = a.act;
  }
  if (a.up) launch_stream<true>(a, act, s);
  else launch_stream<false>(a, act, s);
  return hipGetLastError();
}

}  // namespace moe
