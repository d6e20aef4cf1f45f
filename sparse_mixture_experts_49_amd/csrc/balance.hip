// Balance loss of every sequence of a packed batch, the experts' counts, and the gradient of
// the router's logits.
//
// For sequence b with the n tokens that count (inside its range, not masked out):
//   q_t = softmax(l_t), or s / sum s with s = sigmoid(l_t)
//   load_be = choices of expert e,  mean_be = sum_t q_te / n
//   loss_b = sum_e f_be mean_be,  f_be = E load_be / (k n);  loss = mean over the b with n > 0
// load is a constant in the gradient.  With c_e = d_loss_b E load_be / (k n^2):
//   softmax d l_e = q_e (c_e - sum_j c_j q_j);  sigmoid the same times 1 - s_e
// The difference is formed after the c of an expert with over half of the score is taken off
// every c, so that its own keeps its digits.
//
// Bound by reading the logits (and writing their gradients).  A token is held by L lanes of
// four experts each, L the least power of two with 4 L >= E, so its softmax is a few
// exchanges between neighbouring lanes and a wave works on 64 / L tokens at once.
//
// Sums: a block sums a run of tokens, sequence by sequence.  The pieces (run c, sequence b)
// that are not empty are met in an order in which c or b grows and neither falls, so c + b
// numbers them without gaps in use and without a list.  A second kernel adds each sequence's
// pieces in order, a third the sequences' losses.  fp32 within a piece, fp64 beyond.
//
// 131072 tokens, 256 experts, sigmoid, 64 sequences: 41 us, 3.4 TB/s; runs 34 (28 by bytes at a copy's rate;
// instructions count too: 24 more a token and wave took 2), the two others 5 and 4.  Its gradient 57 us, 4.7 TB/s.
// A small batch: 4.6 and 8 us.
#include <algorithm>
#include <type_traits>

#include "balance.h"
#include "device_common.h"
#include "score.h"

namespace moe {

// Tokens a run has: short runs while there are fewer than 1024 of them, then longer ones, of 512 at
// most, so that a lane's fp32 sum stays short.
static int chunk_of(int T) { return T <= 16 * 1024 ? 16 : std::min(512, (T + 1023) / 1024); }
int balance_chunks(const BalanceShape& s) { const int c = chunk_of(s.T); return (s.T + c - 1) / c; }
int balance_blocks(int E) { return (E + 63) / 64; }

// A lane's four logits of a row (experts e .. e + 3), -inf behind E.  No branches: loads of several
// tokens are to be under way at once.
template <bool VEC>
__device__ __forceinline__ f32x4 load_logits(const float* __restrict__ row, int e, int E) {
  f32x4 v;
  if constexpr (VEC) {
    v = *reinterpret_cast<const f32x4*>(row + min(e, E - 4));
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = row[min(e + j, E - 1)];
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j] = e + (VEC ? 0 : j) < E ? v[j] : -INFINITY;
  return v;
}

// Whether a token counts, likewise: without a mask any byte is read in its place.
struct TokenMask {
  const uint8_t* p;
  bool none;
  __device__ TokenMask(const uint8_t* mask, const float* logits)
      : p(mask ? mask : reinterpret_cast<const uint8_t*>(logits)), none(!mask) {}
  __device__ __forceinline__ bool operator[](int t) const {
    const uint8_t v = p[t];
    return none | (v != 0);
  }
};

// e^x as exp_f32 gives it (2 ulp for |x| < 88; from there without the correction), with two instructions
// less: 2^t of t = x log2 e rounded, times 1 + what x has beyond t ln 2.  Without that the error grows with |x|
// (82 half steps in a share of scores of e^-80).
__device__ __forceinline__ float exp_score(float x) {
  constexpr float kLn2 = 0.69314718055994530942f, kLn2Lo = -1.90465429995776804525e-9f;
  const float t = x * 1.44269504088896340736f, r = __builtin_amdgcn_exp2f(t);
  const float c = fmaf(-t, kLn2Lo, fmaf(-t, kLn2, x));
  return fabsf(x) < 88.f ? fmaf(r, c, r) : r;
}
// 1 / x within 1 ulp, which is 2 of a share's 25 half steps.  (The exact quotient is ten instructions: with it and
// exp_f32 the runs of 131072 x 256 took 36.5 us instead of 34.2, their gradient 60 instead of 57.)
__device__ __forceinline__ float inverse(float x) { return __builtin_amdgcn_rcpf(x); }

// Scores e of a token from its logits and the inverse of their sum, of which q = e inv are the
// shares; REST: for sigmoid scores also 1 - s.
template <int L, bool SIGMOID, bool REST>
__device__ __forceinline__ float scores(const f32x4& l, f32x4& e, f32x4& rest) {
  if constexpr (SIGMOID) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (REST) {
        const float t = exp_score(-fabsf(l[j])), big = inverse(1.f + t), small = t * big;
        e[j] = l[j] < 0.f ? small : big;
        rest[j] = l[j] < 0.f ? big : small;
      } else {
        e[j] = inverse(1.f + exp_score(-l[j]));
      }
    }
  } else {
    float m = lanes_max<L>(fmaxf(fmaxf(l[0], l[1]), fmaxf(l[2], l[3])));
    m = m == -INFINITY ? 0.f : m;                    // every expert masked: no shares
#pragma unroll
    for (int j = 0; j < 4; ++j) e[j] = exp_score(l[j] - m);
  }
  const float sum = lanes_sum<L>((e[0] + e[1]) + (e[2] + e[3]));
  if constexpr (SIGMOID) return inverse(sum < kLeastSum ? kLeastSum : sum);
  return sum > 0.f ? inverse(sum) : sum != sum ? sum : 0.f;
}

// The borders of the sequences, brought into [0, T] and order, so that no content of
// `offsets` leads out of the arrays.
__device__ __forceinline__ int border(const int32_t* __restrict__ offsets, int b, int T) {
  return min(max(offsets[b], 0), T);
}

// The first sequence that ends behind token t (S if none does), 64 of them probed at a time:
// every lane takes part.
__device__ __forceinline__ int sequence_of(const int32_t* __restrict__ offsets, int S, int T, int t) {
  int lo = 0, hi = S;
  while (lo < hi) {
    const int step = (hi - lo + 63) / 64, p = lo + (int)(threadIdx.x & 63) * step + step - 1;
    const uint64_t behind = __ballot(p >= hi || border(offsets, min(p, hi - 1) + 1, T) > t);
    if (!behind) return hi;
    lo += (__ffsll((unsigned long long)behind) - 1) * step;
    hi = min(hi, lo + step - 1);
  }
  return lo;
}

// What a block of four waves holds of a piece: the waves' sums of shares, choices, tokens.
template <int L>
struct PieceSums {
  float q[4][4 * L];
  int hist[kBalanceMaxExperts];
  int count;
  __device__ __forceinline__ void clear(int E) {
    for (int i = threadIdx.x; i < E; i += 256) hist[i] = 0;
    if (threadIdx.x == 0) count = 0;
  }
  __device__ __forceinline__ float share(int e) const { return (q[0][e] + q[1][e]) + (q[2][e] + q[3][e]); }
};

// The sums of tokens [lo, hi) into s, cleared before; complete after a barrier.
template <int L, bool SIGMOID, bool VEC>
__device__ __forceinline__ void sum_piece(const BalanceArgs& a, int lo, int hi, PieceSums<L>& s) {
  constexpr int kTok = 64 / L, kAhead = 4;           // tokens of a wave at once; such steps under way
  const int E = a.sh.E, k = a.sh.k;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int e = (lane % L) * 4, slot = wave * kTok + lane / L;
  const TokenMask mask(a.mask, a.logits);
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  for (int t = lo + slot; t < hi + slot; t += kAhead * 4 * kTok) {      // the same trips for all lanes of a wave
    f32x4 l[kAhead];
    bool in[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int at = min(t + i * 4 * kTok, hi - 1);
      l[i] = load_logits<VEC>(a.logits + (size_t)at * E, e, E);
      in[i] = mask[at] & (t + i * 4 * kTok < hi);
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (!__ballot(in[i])) continue;
      f32x4 q, rest;
      const float inv = scores<L, SIGMOID, false>(l[i], q, rest);
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[j] += in[i] ? q[j] * inv : 0.f;
    }
  }
  int n = 0;
  for (int i = threadIdx.x; i < (hi - lo) * k; i += 256) {
    const int t = lo + i / k, id = a.topk_idx[(size_t)lo * k + i];
    const bool in = mask[t];
    if (in && (uint32_t)id < (uint32_t)E) atomicAdd(&s.hist[id], 1);   // counts: order-independent
    n += in && i % k == 0;
  }
  if (n) atomicAdd(&s.count, n);
#pragma unroll
  for (int o = L; o < 64; o <<= 1)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[j] += __shfl_xor(acc[j], o);
  if (lane < L)
#pragma unroll
    for (int j = 0; j < 4; ++j) s.q[wave][e + j] = acc[j];
}

template <int L, bool SIGMOID, bool VEC>
__global__ __launch_bounds__(256) void balance_part_kernel(BalanceArgs a, int chunk) {
  __shared__ PieceSums<L> s;
  const int T = a.sh.T, E = a.sh.E, S = a.sh.S;
  const int t0 = blockIdx.x * chunk, t1 = min(t0 + chunk, T);
  if (a.total_load && blockIdx.x == 0)
    for (int i = threadIdx.x; i < E; i += 256) a.total_load[i] = 0;
  s.clear(E);
  __syncthreads();
  int empty = 0;                                     // in a row: from two on the next full one is searched for
  for (int b = sequence_of(a.offsets, S, T, t0); b < S; ++b) {
    const int lo = max(border(a.offsets, b, T), t0), hi = min(border(a.offsets, b + 1, T), t1);
    if (lo >= t1) break;
    if (hi <= lo) {
      if (++empty > 1) b = max(b, sequence_of(a.offsets, S, T, lo) - 1);
      continue;
    }
    empty = 0;
    sum_piece<L, SIGMOID, VEC>(a, lo, hi, s);
    __syncthreads();
    const size_t at = (size_t)blockIdx.x + b;
    for (int i = threadIdx.x; i < E; i += 256) {
      a.pq[at * E + i] = s.share(i);
      a.pload[at * E + i] = s.hist[i];
    }
    if (threadIdx.x == 0) a.pvalid[at] = s.count;
    __syncthreads();
    s.clear(E);
    __syncthreads();
  }
}

// A small batch in one launch: a wave has every 16th sequence to itself, no barrier before the end.
template <int L, bool SIGMOID, bool VEC>
__global__ __launch_bounds__(1024) void balance_single_kernel(BalanceArgs a) {
  constexpr int kTok = 64 / L, kAhead = 4, kWaves = 16;
  __shared__ int hist[kWaves][4 * L], all[4 * L], lives[kWaves];
  __shared__ double losses[kWaves];
  const int T = a.sh.T, E = a.sh.E, S = a.sh.S, k = a.sh.k;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int e = (lane % L) * 4, slot = lane / L;
  const TokenMask mask(a.mask, a.logits);
  int* mine = hist[wave];
  if (threadIdx.x < 4 * L) all[threadIdx.x] = 0;
  __syncthreads();
  double total = 0.0;
  int live = 0;
  for (int b = wave; b < S; b += kWaves) {
    const int lo = border(a.offsets, b, T), hi = border(a.offsets, b + 1, T);
    for (int i = lane; i < 4 * L; i += 64) mine[i] = 0;
    f32x4 acc = {0.f, 0.f, 0.f, 0.f};
    int n = 0;
    for (int t = lo + slot; t < hi + slot; t += kAhead * kTok) {
      f32x4 l[kAhead];
      bool in[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int at = min(t + i * kTok, hi - 1);
        l[i] = load_logits<VEC>(a.logits + (size_t)at * E, e, E);
        in[i] = mask[at] & (t + i * kTok < hi);
      }
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        f32x4 q, rest;
        const float inv = scores<L, SIGMOID, false>(l[i], q, rest);
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[j] += in[i] ? q[j] * inv : 0.f;
        n += __popcll(__ballot(in[i] && lane % L == 0));
      }
    }
    for (int i = lane; i < (hi - lo) * k; i += 64) {
      const int id = a.topk_idx[(size_t)lo * k + i];
      if (mask[lo + i / k] && (uint32_t)id < (uint32_t)E) atomicAdd(&mine[id], 1);
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int o = L; o < 64; o <<= 1)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[j] += __shfl_xor(acc[j], o);
    double loss = 0.0;
    if (lane < L)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (e + j < E) {
          const int load = mine[e + j];
          const double mean = n ? (double)acc[j] / n : 0.0;
          loss += n ? (double)E * load / ((double)k * n) * mean : 0.0;
          a.load[(size_t)b * E + e + j] = load;
          if (a.prob_mean) a.prob_mean[(size_t)b * E + e + j] = (float)mean;
          if (load) atomicAdd(&all[e + j], load);
        }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) loss += __shfl_xor(loss, o);
    if (lane == 0) {
      a.valid[b] = n;
      if (a.seq_loss) a.seq_loss[b] = (float)loss;
    }
    total += loss;
    live += n > 0;
  }
  if (lane == 0) losses[wave] = total, lives[wave] = live;
  __syncthreads();
  if (a.total_load && (int)threadIdx.x < E) a.total_load[threadIdx.x] = all[threadIdx.x];
  if (threadIdx.x) return;
#pragma unroll
  for (int w = 1; w < kWaves; ++w) total += losses[w], live += lives[w];
  a.valid[S] = live;
  if (a.loss) *a.loss = live ? (float)(total / live) : 0.f;
}

// A sequence's pieces added up for 64 experts, by W waves: each takes a share of them.
template <int W>
__global__ __launch_bounds__(1024) void balance_seq_kernel(BalanceArgs a, int chunk) {
  __shared__ double sq[16][64];
  __shared__ int sl[16][64], sn[16];
  const int T = a.sh.T, E = a.sh.E, lane = threadIdx.x & 63, wave = threadIdx.x >> 6, e = blockIdx.y * 64 + lane;
  const int b = blockIdx.x * (16 / W) + wave / W, lo = b < a.sh.S ? border(a.offsets, b, T) : 0;
  const int hi = b < a.sh.S ? border(a.offsets, b + 1, T) : 0;
  const int c0 = lo / chunk, c1 = hi > lo ? (hi - 1) / chunk + 1 : c0;
  double q = 0.0;
  int load = 0, n = 0;
#pragma unroll 4
  for (int c = c0 + wave % W; c < c1; c += W) {
    const size_t at = (size_t)c + b;
    if (e < E) {
      q += (double)a.pq[at * E + e];
      load += a.pload[at * E + e];
    }
  }
  for (int c = c0 + wave % W * 64 + lane; c < c1; c += W * 64) n += a.pvalid[(size_t)c + b];
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) n += __shfl_xor(n, o);
  if constexpr (W > 1) {
    sq[wave][lane] = q;
    sl[wave][lane] = load;
    if (lane == 0) sn[wave] = n;
    __syncthreads();
    if (wave % W) return;
#pragma unroll
    for (int w = 1; w < W; ++w) q += sq[wave + w][lane], load += sl[wave + w][lane], n += sn[wave + w];
  }
  if (b >= a.sh.S) return;
  const double mean = n ? q / n : 0.0;
  double part = n && e < E ? (double)E * load / ((double)a.sh.k * n) * mean : 0.0;
  if (e < E) {
    a.load[(size_t)b * E + e] = load;
    if (a.prob_mean) a.prob_mean[(size_t)b * E + e] = (float)mean;
    if (a.total_load && load) atomicAdd(&a.total_load[e], load);
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) part += __shfl_xor(part, o);
  if (lane == 0) {
    a.part[(size_t)b * gridDim.y + blockIdx.y] = part;
    if (blockIdx.y == 0) a.valid[b] = n;
  }
}

// (By the last block of the kernel before it cost more than this launch: every block's release writes
// its L2 back, 64 sequences 44 us against 41, 4096 335 against 105.)
__global__ __launch_bounds__(1024) void balance_total_kernel(BalanceArgs a, int parts) {
  __shared__ double sl[16];
  __shared__ int sn[16];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  double loss = 0.0;
  int live = 0;
  for (int b = threadIdx.x; b < a.sh.S; b += 1024) {
    double l = 0.0;
    for (int p = 0; p < parts; ++p) l += a.part[(size_t)b * parts + p];
    if (a.seq_loss) a.seq_loss[b] = (float)l;
    loss += l;
    live += a.valid[b] > 0;
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) loss += __shfl_xor(loss, o), live += __shfl_xor(live, o);
  if (lane == 0) sl[wave] = loss, sn[wave] = live;
  __syncthreads();
  if (threadIdx.x) return;
#pragma unroll
  for (int w = 1; w < 16; ++w) loss += sl[w], live += sn[w];
  a.valid[a.sh.S] = live;
  if (a.loss) *a.loss = live ? (float)(loss / live) : 0.f;
}

// A wave's tokens are neighbours, so the coefficients change only where a sequence does.
template <int L, bool SIGMOID, bool VEC>
__global__ __launch_bounds__(256) void balance_grad_kernel(BalanceGradArgs a, int per) {
  constexpr int kTok = 64 / L, kAhead = 4;
  const int T = a.sh.T, E = a.sh.E, S = a.sh.S;
  const int lane = threadIdx.x & 63;
  const int e = (lane % L) * 4, slot = lane / L;
  const TokenMask mask(a.mask, a.logits);
  const int w0 = __builtin_amdgcn_readfirstlane((blockIdx.x * 4 + (threadIdx.x >> 6)) * per);
  if (w0 >= T) return;
  const int w1 = min(w0 + per, T);
  const float up = a.d_loss ? *a.d_loss : 0.f;
  const int live_seqs = a.valid[S];
  auto write = [&](int t, const f32x4& d) {
    float* row = a.d_logits + (size_t)t * E;
    if constexpr (VEC) {
      if (e < E) *reinterpret_cast<f32x4*>(row + e) = d;
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (e + j < E) row[e + j] = d[j];
    }
  };
  int at = w0, empty = 0;                            // tokens below are done; empty sequences in a row
  for (int b = sequence_of(a.offsets, S, T, w0); at < w1; ++b) {
    const int lo = b < S ? min(max(border(a.offsets, b, T), at), w1) : w1;
    for (int t = at + slot; t < lo; t += kTok) write(t, f32x4{0.f, 0.f, 0.f, 0.f});   // of no sequence
    if (b >= S) break;
    const int hi = min(max(border(a.offsets, b + 1, T), lo), w1);
    at = hi;
    if (hi <= lo) {
      if (++empty > 1 && at < w1) b = max(b, sequence_of(a.offsets, S, T, at) - 1);
      continue;
    }
    empty = 0;
    f32x4 c;
    const int n = a.valid[b];
    const double by = n > 0 && live_seqs > 0
                          ? ((double)up / live_seqs + (a.d_seq_loss ? (double)a.d_seq_loss[b] : 0.0)) * E /
                                ((double)a.sh.k * n * n)
                          : 0.0;
#pragma unroll
    for (int j = 0; j < 4; ++j) c[j] = e + j < E ? (float)(by * a.load[(size_t)b * E + e + j]) : 0.f;
    for (int t0 = lo + slot; t0 < hi + slot; t0 += kAhead * kTok) {
      f32x4 l[kAhead];
      bool counts[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int row = min(t0 + i * kTok, hi - 1);
        l[i] = load_logits<VEC>(a.logits + (size_t)row * E, e, E);
        counts[i] = mask[row];
      }
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int t = t0 + i * kTok;
        const bool in = counts[i];
        f32x4 q, rest, d;
        const float inv = scores<L, SIGMOID, SIGMOID>(l[i], q, rest);
        float lead = 0.f, dot = 0.f;
        bool leads = false;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          q[j] *= inv;
          leads |= q[j] > 0.5f;
        }
        if (__ballot(leads)) {
#pragma unroll
          for (int j = 0; j < 4; ++j) lead += q[j] > 0.5f ? c[j] : 0.f;
          lead = lanes_sum<L>(lead);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          d[j] = c[j] - lead;
          dot = fmaf(d[j], q[j], dot);
        }
        dot = lanes_sum<L>(dot);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          d[j] = q[j] * (d[j] - dot);
          if (SIGMOID) d[j] *= rest[j];
          d[j] = in ? d[j] : 0.f;
        }
        if (t < hi) write(t, d);
      }
    }
  }
}

// ---- launches ------------------------------------------------------------------------------
template <typename F>
static void for_experts(int E, F f) {
  if (E <= 16) f(std::integral_constant<int, 4>());
  else if (E <= 32) f(std::integral_constant<int, 8>());
  else if (E <= 64) f(std::integral_constant<int, 16>());
  else if (E <= 128) f(std::integral_constant<int, 32>());
  else f(std::integral_constant<int, 64>());
}

template <typename F>
static void for_kind(bool sigmoid, int E, F f) {
  for_experts(E, [&](auto l) {
    auto with = [&](auto s) { E % 4 ? f(l, s, std::false_type()) : f(l, s, std::true_type()); };
    sigmoid ? with(std::true_type()) : with(std::false_type());
  });
}

// Lanes that hold a token.
static int lanes_of(int E) {
  int l = 0;
  for_experts(E, [&](auto n) { l = decltype(n)::value; });
  return l;
}

// One launch where a wave can take a whole sequence: at most 32 of its steps in all, so 512 tokens, and 64
// sequences.  One launch and three, us, 8 experts: 4 sequences of 8 steps 6.6 and 9.4, of 32 steps 15.7 and 9.9;
// 64 of half a step 19.8 and 11.2, with 256 experts 23.6 and 32.5.  A single sequence of 8 steps 6.2 and 9.2, of 16
// 9.1 and 9.3, of 32 15 and 9.5, of 128 50 and 11.6; how long the longest is the host does not know.
static bool single(const BalanceShape& s) { return s.S <= 64 && (long)s.T * lanes_of(s.E) <= 32 * 64; }

hipError_t launch_balance(const BalanceArgs& a, hipStream_t s) {
  if (single(a.sh)) {
    for_kind(a.sh.sigmoid, a.sh.E, [&](auto l, auto sig, auto vec) {
      balance_single_kernel<decltype(l)::value, decltype(sig)::value, decltype(vec)::value><<<1, 1024, 0, s>>>(a);
    });
    return hipGetLastError();
  }
  const int chunk = chunk_of(a.sh.T), parts = balance_blocks(a.sh.E);
  for_kind(a.sh.sigmoid, a.sh.E, [&](auto l, auto sig, auto vec) {
    balance_part_kernel<decltype(l)::value, decltype(sig)::value, decltype(vec)::value>
        <<<balance_chunks(a.sh), 256, 0, s>>>(a, chunk);
  });
  // A sequence's pieces by 16 waves or by one, 131072 x 256, the whole call without total_load: 64 sequences 38
  // and 43 us, 128 37 and 39, 512 42 and 37, 4096 104 and 47.  total_load's atomics meet at E counts: 512
  // sequences 8 us more, 4096 110; 131072 x 64 in 65536 sequences 1390 us with and 197 without it.
  if (balance_chunks(a.sh) >= 8 * a.sh.S) balance_seq_kernel<16><<<dim3(a.sh.S, parts), 1024, 0, s>>>(a, chunk);
  else balance_seq_kernel<1><<<dim3((a.sh.S + 15) / 16, parts), 1024, 0, s>>>(a, chunk);
  balance_total_kernel<<<1, 1024, 0, s>>>(a, parts);
  return hipGetLastError();
}

hipError_t launch_balance_grad(const BalanceGradArgs& a, hipStream_t s) {
  for_kind(a.sh.sigmoid, a.sh.E, [&](auto l, auto sig, auto vec) {
    constexpr int kTok = 64 / decltype(l)::value;
    // 8 steps of a wave each while that gives 8192 waves, more beyond.
    const int per = kTok * std::max(8, (a.sh.T / kTok + 8191) / 8192);
    const int blocks = (a.sh.T + 4 * per - 1) / (4 * per);
    balance_grad_kernel<decltype(l)::value, decltype(sig)::value, decltype(vec)::value><<<blocks, 256, 0, s>>>(a, per);
  });
  return hipGetLastError();
}

}  // namespace moe
