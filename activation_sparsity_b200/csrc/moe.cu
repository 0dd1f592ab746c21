// A mixture-of-experts layer for 1 to 16 tokens in one kernel (sm_100a):
//
//   l[m][e]  = sum_i x[m][i] Wr[e][i]                       router scores
//   S_m      = the k experts of largest l[m] (ties: the lower index)
//   p[m][s]  = softmax over S_m (renormalised), or over every expert
//   h        = silu(x W_gate[e]) * (x W_up[e]),  silu(v) = v / (1 + exp(-v))
//   y[m]     = sum_s p[m][s] (h[m][s] W_down[e_s])
//
// Experts are row-major like every weight of the library: W_gu [E][d][2 f]
// (gate | up along the columns) and W_d [E][f][d], in bf16, fp32 or MX4 with
// blocks down the rows.
//
// Few tokens make it a stream of the chosen experts' weights, bound by HBM
// (bf16: one product per 2 bytes and token), in three steps that depend on one
// another: scores, then gate|up, then down.  As launches of their own the
// boundaries cost a drain, a launch and a ramp each, more than the whole stream
// of a small layer; here one cooperative grid passes four grid-wide barriers
// of about 1.2 us, and a warp asks for its first down rows to be brought into
// L2 before it waits.
//
//   scores   a CTA per expert and four tokens, its warps each a share of the
//            inputs, summed in fp64: selection is a comparison, so scores that
//            differ by less than fp32 rounding must not swap.  (Products of
//            two fp32 values are exact in fp64.)
//   routing  every CTA makes the same selection and the same work list from
//            the scores.  A group is an expert and up to eight of its tokens.
//   products a unit is a group and 128 columns, cut into chunks of rows; a warp
//            takes a unit's chunk as one stream with no barrier in it and
//            writes its sums to the workspace.  How many units there are is
//            known only after the routing, so every CTA chooses the same number
//            of chunks there, the one that ends the last warp first.  Shares lie in
//            the order group, chunk, tile: a CTA's eight warps read the same
//            rows, side by side, and so do the CTAs at work.  With each warp on
//            rows of its own the same bytes took a tenth longer (43 and 38.5 us
//            for 128 bf16 experts of 2048 to 768, 262 and 234 for the 4-bit
//            layer below).
//   joins    after a barrier, the chunks' sums are added in their order: h from
//            gate and up, then y from the experts.  Results repeat bit for bit.
//
// The products run on mma.sync.m16n8k16 with fp32 accumulators: eight tokens
// of fp32 FMAs per 2-byte weight would be the limit instead of HBM.  A lane
// loads 16 bytes (eight columns) of four rows of a 16-row step, so that every
// weight row is read in 128-byte segments, and two byte permutations make
// the A operand's pairs along the reduction; the tokens are the eight columns
// of B.  The bf16 input is its own operand; h, an fp32 value, enters as three
// bf16 pieces (24 significant bits) into the same accumulator, a fresh one for
// every step.  4-bit experts
// use the block products of mx4_mma.cuh, with x and h as two f16 pieces per
// block of 32 that travel through the warp's ring with the rows (loaded
// straight from L2 they held up the stream: 299 and 266 us).  fp32 experts use
// fp32 FMAs on rows that come through a ring as well.
//
// Measured (B200, graph replay, weights from HBM): one token, 8 of 128 bf16
// experts of 2048 to 768, 34.5 us (75 MB, 2.2 TB/s: 13 us outside the two
// streams, which run at 3.6 TB/s); five tokens, 4 of 60 fp32 experts of 1024 to
// 1408, 79 to 83 us (303 MB, 3.7 TB/s, from one placement of the weights to
// another); 16 tokens, 2 of 8 4-bit experts of 4096 to 14336, 234 us (742 MB,
// 3.2 TB/s: bound by issue and mma.sync, the same copies without the products
// take 176 us); a layer of 8 bf16 experts of 256 to 512, 15.6 us, all of it the
// chain of barriers and the first fetch of each phase's code.
#include <algorithm>

#include "common.cuh"
#include "internal.h"
#include "mx4_mma.cuh"

namespace larosa {
namespace {

constexpr int kT = 256;
constexpr int kWarps = kT / 32;
constexpr int kGroup = 8;      // tokens of a group
constexpr int kMaxE = 512;     // LAROSA_MOE_MAX_E
constexpr int kMaxK = 16;      // LAROSA_MOE_MAX_K
constexpr int kMaxPairs = 16 * kMaxK;
constexpr int kMaxRanked = 512;  // scores that are selected by rank
constexpr int kMinShare = 2;    // row steps of a share, at least

enum class Fmt { BF16, F32, MX4 };

// Words of the workspace's zero-filled header: arrivals at the barriers and at
// the end, and shares taken beyond the first of every warp in the two product
// phases.
constexpr int kBarriers = 4, kSyncEnd = kBarriers, kTaken1 = 5, kTaken2 = 6, kSyncWords = 7;

struct MParams {
  const void* x;
  const void* wr;
  const uint8_t* gu;
  const uint8_t* gus;
  const uint8_t* dn;
  const uint8_t* dns;
  float* y;
  int32_t* idx;  // may be null
  float* gate;   // may be null
  unsigned* sync;
  double* logits;        // [M][E]
  unsigned char* xop;    // MX4: x's pieces [M][2][d] f16, then scales [M][d / 32]
  unsigned char* hop;    // h: bf16 pieces [pairs][3][f], fp32 [pairs][f], or as xop
  float* part1;          // [parts][pairs][2 f]
  float* part2;          // [parts][pairs][d]
  int M, d, f, E, k;
  int renormalize;
  int x_f32;             // MX4 experts: x and Wr are fp32
  int* dev_status;
  unsigned long long wait_ns;
};

// How a phase's products are cut into shares for the warps: `units` (a group
// and 128 columns) by `chunks` chunks of `rows` row steps (the last one may be
// shorter).  Shares are taken in the order group, chunk, tile, so that the
// warps at work read whole rows side by side.
struct Cut {
  int units, chunks, rows, shares;

  // The most chunks that are considered: `rounds` shares per warp, of at least
  // kMinShare steps.
  static __host__ __device__ int most(int units, int steps, int workers, int rounds) {
    const int n = rounds * workers / units + 1;
    return n < steps / kMinShare ? n : steps / kMinShare < 1 ? 1 : steps / kMinShare;
  }
  // Time of a phase in row steps: every round of shares costs its rows and a
  // start, and the last share to end may lag by `lag` sixteenths of one.  In
  // floating point, whose divisions take a tenth of the whole numbers' time: a
  // quotient that is a whole number may come out a little larger, hence the
  // offsets (fractions are at least 1 / 2368).
  static __device__ __forceinline__ float cost(int units, int steps, int workers, int c, int start, int lag) {
    const float rows = ceilf(__fdividef((float)steps, (float)c) - 2e-4f);
    const float shares = (float)units * ceilf(__fdividef((float)steps, rows) - 2e-4f);
    const float waves = ceilf(__fdividef(shares, (float)workers) - 2e-4f);
    return 16.f * waves * (rows + (float)start) + (float)lag * rows;
  }
  // By a whole warp.
  __device__ void choose(int units_, int steps, int workers, int rounds, int start, int lag) {
    const int lane = threadIdx.x & 31;
    const int n = most(units_, steps, workers, rounds);
    unsigned best = 0xffffffffu, at = 1;  // costs are positive: their bits compare as they do
#pragma unroll 1
    for (int c = lane + 1; c <= n; c += 32) {
      const unsigned v = __float_as_uint(cost(units_, steps, workers, c, start, lag));
      if (v < best) {
        best = v;
        at = c;
      }
    }
    const unsigned least = __reduce_min_sync(0xffffffffu, best);
    at = __reduce_min_sync(0xffffffffu, best == least ? at : 0xffffffffu);
    if (lane == 0) {
      units = units_;
      rows = (steps + (int)at - 1) / (int)at;
      chunks = (steps + rows - 1) / rows;
      shares = units * chunks;
    }
  }
  // A warp's first share: equally many neighbours for every CTA.
  __device__ __forceinline__ int first(int warp) const {
    const int per = min(kWarps, (shares + (int)gridDim.x - 1) / (int)gridDim.x);
    return warp < per ? (int)blockIdx.x * per + warp : shares;
  }
};

// The routing of a call, the same in every CTA.
struct Routing {
  float gate[kMaxPairs];
  int expert[kMaxPairs];
  short g_expert[kMaxPairs];
  short g_n[kMaxPairs];
  uint8_t g_pair[kMaxPairs][kGroup];
  Cut up, down;  // gate | up, down
  int groups;
  int ok;
};
static_assert(kMaxPairs <= 256, "a pair's number is a byte");

// What the phases without products work in; lies where the products keep
// their rows.
struct Scratch {
  union {
    struct {
      int cnt[kMaxE];
      int base[kMaxE];
    };
    struct {  // selection by rank: the scores' keys
      unsigned hi[kMaxRanked];
      unsigned lo[kMaxRanked];
    };
  };
  int rank[kMaxRanked];     // scores: in their token's order; pairs: among their expert's
  double score[kMaxPairs];  // of the chosen experts
  double sums[kWarps][4];   // scores: the warps' shares
  float4 join[kWarps][32];  // the warps' shares of a sum of parts
};

// ---------------------------------------------------------------- grid-wide barrier

// Every CTA of the (co-resident) grid arrives at *word, which counts up from
// zero; false once the wait limit has passed.
__device__ __forceinline__ bool grid_barrier(unsigned* word, Routing* r, const MParams& p) {
  __syncthreads();
  if (threadIdx.x == 0) {
    atomic_add_release_gpu(word, 1u);
    const unsigned n = gridDim.x;
    unsigned seen;
    bool ok = true;
    unsigned long long t0 = 0;
    for (unsigned it = 0;; ++it) {
      asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(seen) : "l"(word) : "memory");
      if (seen == n) break;  // it stays there until every CTA has passed
      if ((it & 63u) == 63u) {
        const unsigned long long now = global_timer_ns();
        if (t0 == 0) t0 = now;
        if (now - t0 > p.wait_ns) {
          ok = false;
          break;
        }
      }
    }
    r->ok = ok;
    if (!ok) report(p.dev_status, LAROSA_DEV_TIMEOUT);
  }
  __syncthreads();
  return r->ok != 0;
}

// ---------------------------------------------------------------- scores

template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&v)[8]);
template <>
__device__ __forceinline__ void load8<__nv_bfloat16>(const __nv_bfloat16* p, float (&v)[8]) {
  const uint4 u = __ldg(reinterpret_cast<const uint4*>(p));
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
template <>
__device__ __forceinline__ void load8<float>(const float* p, float (&v)[8]) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}

// Tasks (expert, kTok tokens), one CTA each.  Every load of a step is issued
// before the first product, tokens past the last one read the last one's: with
// a test per token the loads came one after the other (5 tokens of 3616 fp32
// inputs 6.6 us, so 3.2).
template <typename T, int kTok>
__device__ void scores(const MParams& p, Scratch* r) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int tg = (p.M + kTok - 1) / kTok;
  const T* x = static_cast<const T*>(p.x);
  const T* wr = static_cast<const T*>(p.wr);
  for (int task = blockIdx.x; task < p.E * tg; task += gridDim.x) {
    const int e = task / tg, m0 = task % tg * kTok;
    const T* w = wr + (size_t)e * p.d;
    const T* row[kTok];
#pragma unroll
    for (int m = 0; m < kTok; ++m) row[m] = x + (size_t)min(m0 + m, p.M - 1) * p.d;
    double acc[kTok] = {};
#pragma unroll 1
    for (int i = threadIdx.x * 8; i < p.d; i += kT * 8) {
      float wv[8], xv[kTok][8];
      load8<T>(w + i, wv);
#pragma unroll
      for (int m = 0; m < kTok; ++m) load8<T>(row[m] + i, xv[m]);
#pragma unroll
      for (int m = 0; m < kTok; ++m)
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[m] = fma((double)wv[j], (double)xv[m][j], acc[m]);
    }
#pragma unroll
    for (int m = 0; m < kTok; ++m) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) acc[m] += __shfl_xor_sync(0xffffffffu, acc[m], o);
      if (lane == 0) r->sums[warp][m] = acc[m];
    }
    __syncthreads();
    if (threadIdx.x < kTok && m0 + (int)threadIdx.x < p.M) {
      double v = r->sums[0][threadIdx.x];
#pragma unroll
      for (int i = 1; i < kWarps; ++i) v += r->sums[i][threadIdx.x];
      __stcg(p.logits + (size_t)(m0 + threadIdx.x) * p.E + e, v);
    }
    __syncthreads();
  }
}
template <typename T>
__device__ __forceinline__ void scores(const MParams& p, Scratch* r) {
  if (p.M == 1)
    scores<T, 1>(p, r);
  else
    scores<T, 4>(p, r);
}

// v of row `lane` of block `b` of token (or pair) m as MX4 pieces: op holds
// [count][n / 32][2][32] f16, then [count][n / 32] scales.
__device__ __forceinline__ void put_pieces(unsigned char* op, int count, int n, int m, int b, float v, int lane) {
  const unsigned top = __reduce_max_sync(0xffffffffu, __float_as_uint(v) & 0x7fffffffu);
  float up, down;
  mx4::piece_scale(top, &up, &down);
  __half p0, p1;
  mx4::split_pieces(v * up, &p0, &p1);
  __half* row = reinterpret_cast<__half*>(op) + (size_t)m * 2 * n + b * 64 + lane;
  row[0] = p0;
  row[32] = p1;
  if (lane == 0) reinterpret_cast<float*>(op + (size_t)count * 4 * n)[(size_t)m * (n / 32) + b] = down;
}

// ---------------------------------------------------------------- routing

// A score's place in the order: larger scores have larger keys, a NaN the
// smallest of all (1); 0 is left for "taken".
__device__ __forceinline__ unsigned long long score_key(double v) {
  if (v != v) return 1ull;
  v += 0.0;  // -0 counts as +0
  const unsigned long long b = (unsigned long long)__double_as_longlong(v);
  return (b >> 63) ? ~b : b | 0x8000000000000000ull;
}

// The score a key was made of (a NaN's comes back as NaN).
__device__ __forceinline__ double key_score(unsigned long long k) {
  if (k == 1ull) return __longlong_as_double(0x7ff8000000000000ll);
  return __longlong_as_double((long long)((k >> 63) ? k & 0x7fffffffffffffffull : ~k));
}

// Token m's experts and gates: lane s < k of a whole warp holds the s-th
// expert and its score; den: the sum of every expert's exponential, taken
// where the gates are not renormalised.
__device__ __forceinline__ void write_gates(const MParams& p, Routing* r, int m, int expert, double score, float den) {
  const int lane = threadIdx.x & 31;
  const double top = __shfl_sync(0xffffffffu, score, 0);
  const float mine = lane < p.k ? expf((float)(score - top)) : 0.f;
  if (p.renormalize) {
    den = mine;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) den += __shfl_xor_sync(0xffffffffu, den, o);
  }
  if (lane < p.k) {
    const int q = m * p.k + lane;
    r->expert[q] = expert;
    r->gate[q] = mine / den;
    if (blockIdx.x == 0) {
      if (p.idx != nullptr) p.idx[q] = expert;
      if (p.gate != nullptr) p.gate[q] = mine / den;
    }
  }
}

// Selection and softmax of token m by one warp; a lane holds kPer scores.
template <int kPer>
__device__ void route_token(const MParams& p, Routing* r, int m) {
  const int lane = threadIdx.x & 31;
  const double* l = p.logits + (size_t)m * p.E;
  unsigned long long key[kPer];
  bool bad = false;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = lane + 32 * i;
    key[i] = 0ull;
    if (e < p.E) {
      const double v = __ldcg(l + e);
      key[i] = score_key(v);
      bad |= !isfinite(v);
    }
  }
  if (__any_sync(0xffffffffu, bad) && lane == 0 && blockIdx.x == 0) report(p.dev_status, LAROSA_DEV_NONFINITE);
  float den = 0.f;
  int expert = 0;  // lane s: the s-th
  if (!p.renormalize) {
    // the sum over every expert, before keys are taken out
    unsigned long long best = 0ull;
#pragma unroll
    for (int i = 0; i < kPer; ++i) best = key[i] > best ? key[i] : best;
    const unsigned mh = __reduce_max_sync(0xffffffffu, (unsigned)(best >> 32));
    const unsigned ml = __reduce_max_sync(0xffffffffu, (unsigned)(best >> 32) == mh ? (unsigned)best : 0u);
    const double top = key_score((unsigned long long)mh << 32 | ml);
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (lane + 32 * i < p.E) den += expf((float)(key_score(key[i]) - top));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) den += __shfl_xor_sync(0xffffffffu, den, o);
  }
  double score = 0.0;  // lane s: the s-th largest
  for (int s = 0; s < p.k; ++s) {
    unsigned long long best = 0ull;
    int at = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (key[i] > best) {
        best = key[i];
        at = i;
      }
    // the largest upper halves, and only where several lanes share them the rest
    const unsigned hi = (unsigned)(best >> 32);
    const unsigned mh = __reduce_max_sync(0xffffffffu, hi);
    const unsigned holders = __ballot_sync(0xffffffffu, hi == mh);
    unsigned ml, e;
    if (__popc(holders) == 1) {
      const int from = __ffs(holders) - 1;
      ml = __shfl_sync(0xffffffffu, (unsigned)best, from);
      e = __shfl_sync(0xffffffffu, (unsigned)(lane + 32 * at), from);
    } else {
      ml = __reduce_max_sync(0xffffffffu, hi == mh ? (unsigned)best : 0u);
      const bool has = hi == mh && (unsigned)best == ml;
      e = __reduce_min_sync(0xffffffffu, has ? (unsigned)(lane + 32 * at) : 0xffffffffu);
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if ((unsigned)(lane + 32 * i) == e) key[i] = 0ull;
    if (lane == s) {
      score = key_score((unsigned long long)mh << 32 | ml);
      expert = (int)e;
    }
  }
  write_gates(p, r, m, expert, score, den);
}

// Selection by the CTA for few scores in all (at most kMaxRanked): an expert's rank
// is the number of its token's experts that come before it.  One pass of
// comparisons spread over all threads, where a warp's k rounds of searching
// for the largest take about 500 clocks each.
__device__ void route_by_rank(const MParams& p, Routing* r, Scratch* w) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int items = p.M * p.E;
  bool bad = false;
  for (int i = tid; i < items; i += kT) {
    const double v = __ldcg(p.logits + i);
    const unsigned long long key = score_key(v);
    w->hi[i] = (unsigned)(key >> 32);
    w->lo[i] = (unsigned)key;
    w->rank[i] = 0;
    bad |= !isfinite(v);
  }
  if (__syncthreads_or(bad) && tid == 0 && blockIdx.x == 0) report(p.dev_status, LAROSA_DEV_NONFINITE);
  // `share` threads per item, each an equal range of the others
  int share = 1;
  while (items * share * 2 <= kT) share *= 2;
  for (int i = tid; i < items * share; i += kT) {
    const int item = i / share, e = item % p.E;
    const unsigned* row = w->hi + item - e;
    const unsigned mine = row[e];
    const int from = i % share * p.E / share, to = (i % share + 1) * p.E / share;
    int before = 0, same = 0;
#pragma unroll 4
    for (int o = from; o < to; ++o) {
      before += row[o] > mine;
      same += row[o] == mine;
    }
    if (same > (from <= e && e < to ? 1 : 0)) {  // others share the upper half
      const unsigned* low = w->lo + item - e;
      for (int o = from; o < to; ++o) before += row[o] == mine && (low[o] > low[e] || (low[o] == low[e] && o < e));
    }
    if (share == 1)
      w->rank[item] = before;
    else
      atomicAdd(&w->rank[item], before);
  }
  __syncthreads();
  for (int i = tid; i < items; i += kT) {
    const int rank = w->rank[i], m = i / p.E;
    if (rank < p.k) {
      r->expert[m * p.k + rank] = i % p.E;
      w->score[m * p.k + rank] = key_score((unsigned long long)w->hi[i] << 32 | w->lo[i]);
    }
  }
  __syncthreads();
  for (int m = warp; m < p.M; m += kWarps) {
    const int expert = lane < p.k ? r->expert[m * p.k + lane] : 0;
    const double score = lane < p.k ? w->score[m * p.k + lane] : 0.0;
    float den = 0.f;
    if (!p.renormalize) {
      const double top = __shfl_sync(0xffffffffu, score, 0);
      for (int e = lane; e < p.E; e += 32) den += expf((float)(key_score((unsigned long long)w->hi[m * p.E + e] << 32 | w->lo[m * p.E + e]) - top));
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) den += __shfl_xor_sync(0xffffffffu, den, o);
    }
    write_gates(p, r, m, expert, score, den);
  }
  __syncthreads();  // the keys are used up
}

// The groups of up to 32 pairs (token, slot), by one warp: experts in the
// order of their first pair, an expert's pairs in ascending order, eight to a
// group.
__device__ void build_groups_warp(const MParams& p, Routing* r) {
  const int lane = threadIdx.x & 31;
  const int pairs = p.M * p.k;
  const int e = lane < pairs ? r->expert[lane] : -1;
  const unsigned same = __match_any_sync(0xffffffffu, e);
  const int rank = __popc(same & ((1u << lane) - 1u)), cnt = __popc(same);
  const int n = lane < pairs && rank == 0 ? (cnt + kGroup - 1) / kGroup : 0;
  int incl = n;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  const int base = __shfl_sync(0xffffffffu, incl - n, __ffs(same) - 1);
  if (lane < pairs) {
    const int g = base + rank / kGroup;
    r->g_pair[g][rank % kGroup] = (uint8_t)lane;
    if (rank % kGroup == 0) {
      r->g_expert[g] = (short)e;
      r->g_n[g] = (short)min(kGroup, cnt - rank);
    }
  }
  if (lane == 31) r->groups = incl;
}

// The groups of more pairs, by one warp, 32 pairs at a time: experts in ascending
// order.  (Loops are not unrolled here: code that runs once costs more to fetch
// than to run, 3.2 us for 112 pairs with both loops unrolled.)
__device__ void build_groups(const MParams& p, Routing* r, Scratch* w) {
  const int lane = threadIdx.x & 31;
  const int pairs = p.M * p.k;
  for (int e = lane; e < p.E; e += 32) w->cnt[e] = 0;
  __syncwarp();
#pragma unroll 1
  for (int q = lane; q < (pairs + 31) / 32 * 32; q += 32) {
    const int e = q < pairs ? r->expert[q] : -1;
    const unsigned same = __match_any_sync(0xffffffffu, e);
    const int before = e < 0 ? 0 : w->cnt[e], here = __popc(same & ((1u << lane) - 1u));
    __syncwarp();
    if (e >= 0 && here == 0) w->cnt[e] = before + __popc(same);
    __syncwarp();
    w->rank[q] = before + here;
  }
  int groups = 0;
  for (int e0 = 0; e0 < p.E; e0 += 32) {
    const int e = e0 + lane;
    const int n = e < p.E ? (w->cnt[e] + kGroup - 1) / kGroup : 0;
    int incl = n;
#pragma unroll 1
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    if (e < p.E) w->base[e] = groups + incl - n;
    groups += __shfl_sync(0xffffffffu, incl, 31);
  }
  if (lane == 0) r->groups = groups;
  __syncwarp();
#pragma unroll 1
  for (int q = lane; q < pairs; q += 32) {
    const int e = r->expert[q], rank = w->rank[q], g = w->base[e] + rank / kGroup;
    r->g_pair[g][rank % kGroup] = (uint8_t)q;
    if (rank % kGroup == 0) {
      r->g_expert[g] = (short)e;
      r->g_n[g] = (short)min(kGroup, w->cnt[e] - rank);
    }
  }
}

// ---------------------------------------------------------------- products

// A warp's part of a unit: rows [k0, k1) of a matrix with `rows` rows and `ld`
// columns, `width` columns (at most 128) from `col` on.
struct Unit {
  const uint8_t* W;       // the expert's matrix (MX4: codes)
  const uint8_t* scales;  // MX4
  int rows, ld;
  int col, width;
  int k0, k1;
  int n;  // tokens
};

// MX4: a block of 32 rows by 128 columns and the operands of up to eight
// tokens for it.  Token m's 16-byte chunk c (piece, step, half step) lies at
// chunk c ^ 2 (m % 4): four tokens' reads of 32 bytes fall into different banks.
struct __align__(16) Stage {
  mx4::Tile tile;
  __half op[kGroup][2][32];
  float scale[kGroup];

  __device__ __forceinline__ __half* chunk(int m, int c) { return &op[m][0][0] + 8 * (c ^ (2 * (m & 3))); }
};

// fp32: eight rows by 128 columns and the operands of up to eight tokens for them.
struct __align__(16) RowStage {
  float row[8][128];
  float op[kGroup][8];
};

template <Fmt F>
struct Cfg {
  static constexpr int kStep = F == Fmt::BF16 ? 16 : F == Fmt::F32 ? 8 : 32;  // rows of a step
  // For Cut: shares per warp at most, row steps that starting a share takes, and
  // sixteenths of a share that the last may lag.  4-bit shares take longer with
  // more tokens, so several to a warp even them out (16 tokens of 8 experts of
  // 4096 to 14336: at most three 247 us, five 234, eight 244); bf16 and fp32
  // shares wait for HBM, and every further start costs more than it evens out
  // (one token, 128 experts of 2048 to 768: up to two 35.1 us, up to three 38.8).
  static constexpr int kRounds = F == Fmt::MX4 ? 5 : 2;
  static constexpr int kStart = F == Fmt::MX4 ? 2 : 1;
  static constexpr int kLag = F == Fmt::MX4 ? 12 : 4;
  // CTAs per SM.  With one, bf16 products have the registers for two steps of
  // 4 KB in flight per warp while a third is multiplied, and the barriers half as
  // many arrivals (one token, 128 experts: 38.6 us with two CTAs, 35.1 with one;
  // fp32 80 and 82, 4-bit 235 and 245).
  static constexpr int kCtas = F == Fmt::BF16 ? 1 : 2;
  static constexpr int kRing = 3;  // fp32, MX4: stages of a warp's ring
  static constexpr size_t kWarpSmem = F == Fmt::BF16  ? 0
                                      : F == Fmt::F32 ? kRing * sizeof(RowStage)
                                                      : kRing * sizeof(Stage);
  static constexpr size_t kSmem = std::max(kWarps * kWarpSmem, sizeof(Scratch));
};

// Asynchronous copies to shared memory of `bytes` (all or none) bytes; the rest
// is filled with zeros.  By way of L1: the warps of a CTA mostly work on the
// same rows, so that seven of eight find their operand there.
__device__ __forceinline__ void copy16_or_zero(void* dst, const void* src, unsigned bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy4_or_zero(void* dst, const void* src, unsigned bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(bytes) : "memory");
}

// d = A B, or d += A B.
__device__ __forceinline__ void mma_bf16(float (&d)[4], bool fresh, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint2 b) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %11, %12, %13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b.x), "r"(b.y), "f"(fresh ? 0.f : d[0]), "f"(fresh ? 0.f : d[1]),
        "f"(fresh ? 0.f : d[2]), "f"(fresh ? 0.f : d[3]));
}

// bf16 weights.  The operand of the token in column g of B is P rows of
// u.rows bf16 values at `op` (null: no token); o0, o1: where the sums of tokens
// 2 t and 2 t + 1 go (null: nowhere).  A step's products, the smallest pieces
// first, go to a fresh accumulator that is then added to the fp32 sum: the
// tensor cores truncate their additions, which over a whole share puts sums of
// like signs low (on average by 1.6e-7 of themselves at 2048 inputs, where this leaves
// 1e-9; the same times: 34.6 and 34.5 us, one token of 128 experts).
template <int P>
__device__ __forceinline__ void product_bf16(const Unit& u, const __nv_bfloat16* op, float* o0, float* o1) {
  const int lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  // columns 8 g and 64 + 8 g of the unit
  const bool inA = 8 * g < u.width, inB = 64 + 8 * g < u.width;
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  const uint32_t row_bytes = (uint32_t)u.ld * 2;
  const uint8_t* base = u.W + (size_t)(4 * t) * row_bytes;
  const uint32_t offA = (uint32_t)(u.col + 8 * g) * 2, offB = offA + 128;
  float acc[2][4][4] = {};
  struct Rows {
    uint4 w[2][4];
    uint2 b[P];
  };
  auto load = [&](int r0, Rows& s) {
    const bool in = r0 + 4 * t < u.k1;  // rows are multiples of four
    const uint8_t* at = base + (size_t)r0 * row_bytes;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      s.w[0][i] = in && inA ? __ldcs(reinterpret_cast<const uint4*>(at + (size_t)i * row_bytes + offA)) : zero;
      s.w[1][i] = in && inB ? __ldcs(reinterpret_cast<const uint4*>(at + (size_t)i * row_bytes + offB)) : zero;
    }
#pragma unroll
    for (int q = 0; q < P; ++q)
      s.b[q] = in && op != nullptr ? *reinterpret_cast<const uint2*>(op + (size_t)q * u.rows + r0 + 4 * t)
                                   : make_uint2(0u, 0u);
  };
  auto multiply = [&](const Rows& s) {
#pragma unroll
    for (int seg = 0; seg < 2; ++seg)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          w[i] = q == 0 ? s.w[seg][i].x : q == 1 ? s.w[seg][i].y : q == 2 ? s.w[seg][i].z : s.w[seg][i].w;
        const uint32_t a0 = __byte_perm(w[0], w[1], 0x5410), a1 = __byte_perm(w[0], w[1], 0x7632);
        const uint32_t a2 = __byte_perm(w[2], w[3], 0x5410), a3 = __byte_perm(w[2], w[3], 0x7632);
        float d[4];
#pragma unroll
        for (int c = P - 1; c >= 0; --c) mma_bf16(d, c == P - 1, a0, a1, a2, a3, s.b[c]);
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[seg][q][i] += d[i];
      }
  };
  // three steps in turn, two of them on their way while one is multiplied
  Rows s0, s1, s2;
  int r = u.k0;
  load(r, s0);
  if (r + 16 < u.k1) load(r + 16, s1);
  while (true) {
    if (r + 32 < u.k1) load(r + 32, s2);
    multiply(s0);
    if ((r += 16) >= u.k1) break;
    if (r + 32 < u.k1) load(r + 32, s0);
    multiply(s1);
    if ((r += 16) >= u.k1) break;
    if (r + 32 < u.k1) load(r + 32, s1);
    multiply(s2);
    if ((r += 16) >= u.k1) break;
  }
#pragma unroll
  for (int seg = 0; seg < 2; ++seg) {
    if (!(seg == 0 ? inA : inB)) continue;
    const int c = u.col + 64 * seg + 8 * g;
#pragma unroll
    for (int q = 0; q < 4; q += 2) {
      if (o0 != nullptr)
        __stcg(reinterpret_cast<float4*>(o0 + c + 2 * q),
               make_float4(acc[seg][q][0], acc[seg][q][2], acc[seg][q + 1][0], acc[seg][q + 1][2]));
      if (o1 != nullptr)
        __stcg(reinterpret_cast<float4*>(o1 + c + 2 * q),
               make_float4(acc[seg][q][1], acc[seg][q][3], acc[seg][q + 1][1], acc[seg][q + 1][3]));
    }
  }
}

// fp32 weights: eight rows at a time, with their operands, through the warp's
// ring of stages; a lane holds four columns.  mine: operand of token lane / 2 of
// the group, its first row's (null: no token); out(m): where the sums of token m
// go (null: nowhere).  (Rows in registers, eight in flight and eight being
// multiplied, and operands loaded every 32 rows: 264 us where this takes 223, 16
// tokens on 7 of 17 experts of 768 to 5184.)
template <int N, typename Out>
__device__ __forceinline__ void product_f32(const Unit& u, const float* mine, Out out, RowStage* ring) {
  constexpr int kRing = Cfg<Fmt::F32>::kRing;
  const int lane = threadIdx.x & 31;
  const bool in = 4 * lane < u.width;
  const int col = u.col + 4 * lane, half = lane & 1;
  const float* at = reinterpret_cast<const float*>(u.W) + (size_t)u.k0 * u.ld + col;
  const int steps = (u.k1 - u.k0) / 8;
  const unsigned present = mine != nullptr;
  mine = present ? mine + u.k0 + 4 * half : reinterpret_cast<const float*>(u.W);  // else copies of no bytes: zeros
  auto fetch = [&](RowStage& st) {
    if (in) {
#pragma unroll
      for (int i = 0; i < 8; ++i) mx4::copy16_l2(&st.row[i][4 * lane], at + (size_t)i * u.ld);
    }
    if (lane < 2 * N) copy16_or_zero(&st.op[lane >> 1][4 * half], mine, present * 16);
    at += (size_t)8 * u.ld;
    mine += present * 8;
  };
  float acc[N][4] = {};
  __syncwarp();  // the part before has read its stages
#pragma unroll
  for (int s = 0; s < kRing - 1; ++s) {
    if (s < steps) fetch(ring[s]);
    mx4::copies_commit();
  }
  int now = 0, fill = kRing - 1;
#pragma unroll 1
  for (int i = 0; i < steps; ++i) {
    __syncwarp();  // every lane has read the stage that is filled next
    if (i + kRing - 1 < steps) fetch(ring[fill]);
    mx4::copies_commit();
    mx4::copies_wait<kRing - 1>();
    __syncwarp();  // the other lanes' copies too
    const RowStage& st = ring[now];
    now = now + 1 == kRing ? 0 : now + 1;
    fill = fill + 1 == kRing ? 0 : fill + 1;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float4 w[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) w[r] = *reinterpret_cast<const float4*>(&st.row[4 * h + r][4 * lane]);
#pragma unroll
      for (int m = 0; m < N; ++m) {
        const float4 c = *reinterpret_cast<const float4*>(&st.op[m][4 * h]);
        const float v[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          acc[m][0] = fmaf(v[r], w[r].x, acc[m][0]);
          acc[m][1] = fmaf(v[r], w[r].y, acc[m][1]);
          acc[m][2] = fmaf(v[r], w[r].z, acc[m][2]);
          acc[m][3] = fmaf(v[r], w[r].w, acc[m][3]);
        }
      }
    }
  }
  mx4::copies_wait<0>();
  if (!in) return;
#pragma unroll
  for (int m = 0; m < N; ++m) {
    float* const to = out(m);
    if (to != nullptr)
      __stcg(reinterpret_cast<float4*>(to + col), make_float4(acc[m][0], acc[m][1], acc[m][2], acc[m][3]));
  }
}

// MX4 weights: blocks of 32 rows, with their operands, through the warp's ring
// of stages.  mine: pieces and block scales of token lane / 4 of the group, its
// first row's (null: no token).  B holds, in column g:
//   kEight   one piece of token g; o: where the sums of 2 t and 2 t + 1 go
//   else     piece g % 2 of token g / 2; o[0]: of token t
// Null: no token.
template <bool kEight>
__device__ __forceinline__ void product_mx4(const Unit& u, const __half* mine, const float* mine_scales,
                                            float* const (&o)[2], Stage* ring) {
  constexpr int kRing = Cfg<Fmt::MX4>::kRing;
  const int lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int first = u.k0 / 32, blocks = (u.k1 - u.k0) / 32;
  mx4::BlockCopies copies;
  copies.start(u.W, u.scales, u.ld, u.col, u.width, first, 1, lane);
  const unsigned present = mine != nullptr;
  if (present) {
    mine += first * 64 + 16 * t;
    mine_scales += first;
  } else {  // copies of no bytes: zeros
    mine = reinterpret_cast<const __half*>(u.W);
    mine_scales = reinterpret_cast<const float*>(u.W);
  }
  auto fetch = [&](Stage& st) {
    copies.next(st.tile, lane);
    if (kEight || g < 4) {
      copy16_or_zero(st.chunk(g, 2 * t), mine, present * 16);
      copy16_or_zero(st.chunk(g, 2 * t + 1), mine + 8, present * 16);
      if (t == 0) copy4_or_zero(&st.scale[g], mine_scales, present * 4);
    }
    mine += present * 64;
    mine_scales += present;
  };
  __syncwarp();  // the part before has read its stages
#pragma unroll
  for (int s = 0; s < kRing - 1; ++s) {
    if (s < blocks) fetch(ring[s]);
    mx4::copies_commit();
  }
  unsigned long long acc8[1][16];
  float acc4[1][8][2];
#pragma unroll
  for (int c = 0; c < 16; ++c) {
    acc8[0][c] = 0ull;
    acc4[0][c / 2][c % 2] = 0.f;
  }
  int now = 0, fill = kRing - 1;
#pragma unroll 1
  for (int i = 0; i < blocks; ++i) {
    __syncwarp();  // every lane has read the stage that is filled next
    if (i + kRing - 1 < blocks) fetch(ring[fill]);
    mx4::copies_commit();
    mx4::copies_wait<kRing - 1>();
    __syncwarp();  // the other lanes' copies too
    Stage& st = ring[now];
    mx4::RowSet rs;
    rs.read<4, 4>(st.tile, g, t);
    now = now + 1 == kRing ? 0 : now + 1;
    fill = fill + 1 == kRing ? 0 : fill + 1;
    // the four halves of `step` that this lane multiplies, of a token's piece
    auto operand = [&](int m, int piece, int step) {
      return *reinterpret_cast<const uint2*>(st.chunk(m, 4 * piece + 2 * step + (t >> 1)) + 4 * (t & 1));
    };
    if constexpr (kEight) {
      const uint2 b[2][1][2] = {{{operand(g, 0, 0), operand(g, 1, 0)}}, {{operand(g, 0, 1), operand(g, 1, 1)}}};
      const unsigned long long s2[1] = {*reinterpret_cast<const unsigned long long*>(&st.scale[2 * t])};
      mx4::block_product8<1>(rs, b, s2, acc8);
    } else {
      const uint2 b[2][1] = {{operand(g >> 1, g & 1, 0)}, {operand(g >> 1, g & 1, 1)}};
      const float s1[1] = {st.scale[t]};
      mx4::block_product<1, 4, 4>(rs, b, s1, acc4);
    }
  }
  mx4::copies_wait<0>();
  if (16 * g >= u.width) return;
#pragma unroll
  for (int c = 0; c < 16; c += 4) {
    const int col = u.col + 16 * g + c;
    if constexpr (kEight) {
      const float2 v[4] = {mx4::unpack2(acc8[0][c]), mx4::unpack2(acc8[0][c + 1]), mx4::unpack2(acc8[0][c + 2]),
                           mx4::unpack2(acc8[0][c + 3])};
      if (o[0] != nullptr) __stcg(reinterpret_cast<float4*>(o[0] + col), make_float4(v[0].x, v[1].x, v[2].x, v[3].x));
      if (o[1] != nullptr) __stcg(reinterpret_cast<float4*>(o[1] + col), make_float4(v[0].y, v[1].y, v[2].y, v[3].y));
    } else if (o[0] != nullptr) {
      const int q = c / 2;
      __stcg(reinterpret_cast<float4*>(o[0] + col),
             make_float4(acc4[0][q][0], acc4[0][q][1], acc4[0][q + 1][0], acc4[0][q + 1][1]));
    }
  }
}

// A warp's part of a unit of `group`; the pairs' sums go to rows of `ld_out`
// floats at out.  Operand of a pair: x's (gate | up: token q / k) or h's (down:
// pair q).
template <Fmt F, bool kDown>
__device__ __forceinline__ void part_product(const MParams& p, const Routing* r, int group, const Unit& u, float* out,
                                             int ld_out, unsigned char* smem) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int rows = u.rows;
  auto pair_of = [&](int pos) -> int { return pos < u.n ? r->g_pair[group][pos] : -1; };
  auto operand = [&](int pos) -> int {  // row of the operand of the group's pos-th pair, -1: none
    const int q = pair_of(pos);
    return q < 0 || kDown ? q : q / p.k;
  };
  auto sums_of = [&](int pos) -> float* {
    const int q = pair_of(pos);
    return q < 0 ? nullptr : out + (size_t)q * ld_out;
  };
  if constexpr (F == Fmt::BF16) {
    const int o = operand(g);
    float* o0 = sums_of(2 * t);
    float* o1 = sums_of(2 * t + 1);
    if constexpr (kDown)
      product_bf16<3>(u, o < 0 ? nullptr : reinterpret_cast<const __nv_bfloat16*>(p.hop) + (size_t)o * 3 * rows, o0, o1);
    else
      product_bf16<1>(u, o < 0 ? nullptr : static_cast<const __nv_bfloat16*>(p.x) + (size_t)o * rows, o0, o1);
  } else if constexpr (F == Fmt::F32) {
    const float* src = kDown ? reinterpret_cast<const float*>(p.hop) : static_cast<const float*>(p.x);
    const int o = lane < 2 * kGroup ? operand(lane >> 1) : -1;
    const float* mine = o < 0 ? nullptr : src + (size_t)o * rows;
    RowStage* ring = reinterpret_cast<RowStage*>(smem + warp * Cfg<F>::kWarpSmem);
    if (u.n <= 1)
      product_f32<1>(u, mine, sums_of, ring);
    else if (u.n <= 2)
      product_f32<2>(u, mine, sums_of, ring);
    else if (u.n <= 4)
      product_f32<4>(u, mine, sums_of, ring);
    else
      product_f32<8>(u, mine, sums_of, ring);
  } else {
    const unsigned char* src = kDown ? p.hop : p.xop;
    const __half* pieces = reinterpret_cast<const __half*>(src);
    const float* scales = reinterpret_cast<const float*>(src + (size_t)(kDown ? p.M * p.k : p.M) * 4 * rows);
    Stage* ring = reinterpret_cast<Stage*>(smem + warp * Cfg<F>::kWarpSmem);
    const int o = operand(g);
    const __half* mine = o < 0 ? nullptr : pieces + (size_t)o * 2 * rows;
    const float* mine_scales = o < 0 ? nullptr : scales + (size_t)o * (rows / 32);
    if (u.n <= 4) {
      float* const to[2] = {sums_of(t), nullptr};
      product_mx4<false>(u, mine, mine_scales, to, ring);
    } else {
      float* const to[2] = {sums_of(2 * t), sums_of(2 * t + 1)};
      product_mx4<true>(u, mine, mine_scales, to, ring);
    }
  }
}

// h of pair q, columns j .. j + 3 (in: there are such): stored as the operand of
// the down product.  Eight neighbouring lanes hold a block of 32.
template <Fmt F>
__device__ __forceinline__ void put_h(const MParams& p, int q, int j, float4 g, float4 u, bool in) {
  const float a[4] = {g.x, g.y, g.z, g.w}, b[4] = {u.x, u.y, u.z, u.w};
  float h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = a[i] / (1.f + expf(-a[i])) * b[i];
  if constexpr (F == Fmt::BF16) {
    if (!in) return;
    __nv_bfloat16* at = reinterpret_cast<__nv_bfloat16*>(p.hop) + (size_t)q * 3 * p.f + j;
#pragma unroll
    for (int piece = 0; piece < 3; ++piece) {
      __align__(8) __nv_bfloat16 v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[i] = __float2bfloat16_rn(h[i]);
        h[i] -= __bfloat162float(v[i]);
      }
      *reinterpret_cast<uint2*>(at + (size_t)piece * p.f) = *reinterpret_cast<const uint2*>(v);
    }
  } else if constexpr (F == Fmt::F32) {
    if (in) *reinterpret_cast<float4*>(reinterpret_cast<float*>(p.hop) + (size_t)q * p.f + j) = make_float4(h[0], h[1], h[2], h[3]);
  } else {
    unsigned top = 0u;
#pragma unroll
    for (int i = 0; i < 4; ++i) top = max(top, __float_as_uint(h[i]) & 0x7fffffffu);
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (!in) return;  // f is a multiple of 32: whole blocks
    float up, down;
    mx4::piece_scale(top, &up, &down);
    __align__(8) __half v0[4], v1[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) mx4::split_pieces(h[i] * up, &v0[i], &v1[i]);
    __half* at = reinterpret_cast<__half*>(p.hop) + (size_t)q * 2 * p.f + j / 32 * 64 + j % 32;
    *reinterpret_cast<uint2*>(at) = *reinterpret_cast<const uint2*>(v0);
    *reinterpret_cast<uint2*>(at + 32) = *reinterpret_cast<const uint2*>(v1);
    if (j % 32 == 0)
      reinterpret_cast<float*>(p.hop + (size_t)p.M * p.k * 4 * p.f)[(size_t)q * (p.f / 32) + j / 32] = down;
  }
}

// The next share of a warp beyond its first: asked for before the present one
// is worked on (lane 0 holds the answer until then).
__device__ __forceinline__ unsigned ask_share(unsigned* taken) {
  return (threadIdx.x & 31) == 0 ? atomicAdd(taken, 1u) : 0u;
}

__device__ __forceinline__ float4 add4(float4 a, float4 b) {
  return make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w);
}

// Sum of four columns' parts [i0, i1), `step` floats apart, in order.
__device__ __forceinline__ float4 add_parts(const float* from, size_t step, int i0, int i1) {
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  from += (size_t)i0 * step;
  for (int i = i0; i < i1; i += 8, from += 8 * step) {
    float4 v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
      v[j] = i + j < i1 ? __ldcg(reinterpret_cast<const float4*>(from + (size_t)j * step)) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int j = 0; j < 8; ++j) s = add4(s, v[j]);
  }
  return s;
}

template <Fmt F>
__device__ __forceinline__ size_t row_bytes_of(int cols) {
  return F == Fmt::BF16 ? (size_t)cols * 2 : F == Fmt::F32 ? (size_t)cols * 4 : (size_t)cols / 2;
}

// The down rows that a share starts with, on their way to L2.
template <Fmt F>
__device__ __forceinline__ void prefetch_rows(const Unit& u, int lane) {
  const size_t row = row_bytes_of<F>(u.ld), c0 = row_bytes_of<F>(u.col), width = row_bytes_of<F>(u.width);
  const int lines = (int)((width + 127) / 128);
  for (int i = lane; i < (u.k1 - u.k0) * lines; i += 32) {
    const uint8_t* from = u.W + (size_t)(u.k0 + i / lines) * row + c0 + min((size_t)(i % lines) * 128, width - 1);
    asm volatile("prefetch.global.L2 [%0];" ::"l"(from));
  }
}

template <Fmt F>
__global__ void __launch_bounds__(kT, Cfg<F>::kCtas) moe_kernel(const MParams p) {
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ Routing r;
  constexpr int kStep = Cfg<F>::kStep;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int pairs = p.M * p.k;
  // shares are dealt over the CTAs first, so that few of them land on many SMs
  const int me = warp * gridDim.x + blockIdx.x, workers = kWarps * gridDim.x;

  Scratch& work = *reinterpret_cast<Scratch*>(smem);
  pdl_wait();
  pdl_launch_dependents();

  // ------------------------------------------------------------------ scores
  const bool x_f32 = F == Fmt::F32 || (F == Fmt::MX4 && p.x_f32);
  if (x_f32)
    scores<float>(p, &work);
  else
    scores<__nv_bfloat16>(p, &work);
  if constexpr (F == Fmt::MX4) {
    const int blocks = p.d / 32;
    for (int i = me; i < p.M * blocks; i += workers) {
      const int m = i / blocks, b = i % blocks;
      const size_t at = (size_t)m * p.d + b * 32 + lane;
      const float v = x_f32 ? static_cast<const float*>(p.x)[at]
                            : __bfloat162float(static_cast<const __nv_bfloat16*>(p.x)[at]);
      put_pieces(p.xop, p.M, p.d, m, b, v, lane);
    }
  }
  if (!grid_barrier(p.sync, &r, p)) return;

  // ------------------------------------------------------------------ routing
  // Ranks cost M E^2 comparisons over the CTA, rounds k searches for each of the
  // tokens a warp has.  One token of 128 experts, k = 8, gains 0.5 us by ranks and
  // one of 75, k = 6, 0.4; one of 8, k = 2, loses 0.5, five of 60, k = 4, 2.5 and
  // five of 143, k = 4, 5.
  if (p.k >= 4 && p.M * p.E <= kMaxRanked && p.M * p.E * p.E <= 4096 * p.k * ((p.M + kWarps - 1) / kWarps)) {
    route_by_rank(p, &r, &work);
  } else {
    for (int m = warp; m < p.M; m += kWarps) {
      if (p.E <= 32)
        route_token<1>(p, &r, m);
      else if (p.E <= 128)
        route_token<4>(p, &r, m);
      else
        route_token<kMaxE / 32>(p, &r, m);
    }
    __syncthreads();
  }
  if (warp == 0) {
    if (pairs <= 32)
      build_groups_warp(p, &r);
    else
      build_groups(p, &r, &work);
  }
  __syncthreads();
  const int G = r.groups;

  // ------------------------------------------------------------------ gate | up
  // units: tile, group and half (gate, up), the last fastest
  const int up_tiles = (p.f + 127) / 128, down_tiles = (p.d + 127) / 128;
  if (warp < 2) {
    const bool first = warp == 0;
    Cut& cut = first ? r.up : r.down;
    cut.choose(G * (first ? 2 * up_tiles : down_tiles), ((first ? p.d : p.f) + kStep - 1) / kStep, workers,
               Cfg<F>::kRounds, Cfg<F>::kStart, Cfg<F>::kLag);
  }
  __syncthreads();
  const Cut& up = r.up;
  const Cut& down = r.down;
  const size_t up_slab = (size_t)pairs * 2 * p.f;
  const size_t up_bytes = row_bytes_of<F>(2 * p.f) * p.d;
  // shares taken beyond the first of every warp are handed out in order
  const int up_first = up.first(warp), up_taken = min(up.shares, kWarps * (int)gridDim.x);
  for (int share = up_first; share < up.shares;) {
    const unsigned next = ask_share(p.sync + kTaken1);
    const int column = share % (2 * up_tiles), rest = share / (2 * up_tiles);
    const int chunk = rest % up.chunks, group = rest / up.chunks;
    const int half = column >= up_tiles, tile = column - half * up_tiles;
    const int e = r.g_expert[group];
    Unit u;
    u.W = p.gu + (size_t)e * up_bytes;
    u.scales = F == Fmt::MX4 ? p.gus + (size_t)e * (p.d / 32) * (2 * p.f) : nullptr;
    u.rows = p.d;
    u.ld = 2 * p.f;
    u.col = tile * 128 + half * p.f;
    u.width = min(128, p.f - tile * 128);
    u.n = r.g_n[group];
    u.k0 = chunk * up.rows * kStep;
    u.k1 = min(p.d, u.k0 + up.rows * kStep);
    part_product<F, false>(p, &r, group, u, p.part1 + (size_t)chunk * up_slab, 2 * p.f, smem);
    share = up_taken + (int)__shfl_sync(0xffffffffu, next, 0);
  }

  // ------------------------------------------------------------------ down
  const size_t down_slab = (size_t)pairs * p.d;
  const size_t down_bytes = row_bytes_of<F>(p.d) * p.f;
  int share = down.first(warp);
  const int down_taken = min(down.shares, kWarps * (int)gridDim.x);
  auto make_unit = [&](int* group, int* chunk) {
    const int tile = share % down_tiles, rest = share / down_tiles;
    *chunk = rest % down.chunks;
    *group = rest / down.chunks;
    const int e = r.g_expert[*group];
    Unit u;
    u.W = p.dn + (size_t)e * down_bytes;
    u.scales = F == Fmt::MX4 ? p.dns + (size_t)e * (p.f / 32) * p.d : nullptr;
    u.rows = p.f;
    u.ld = p.d;
    u.col = tile * 128;
    u.width = min(128, p.d - u.col);
    u.n = r.g_n[*group];
    u.k0 = *chunk * down.rows * kStep;
    u.k1 = min(p.f, u.k0 + down.rows * kStep);
    return u;
  };
  int group, chunk;
  if (share < down.shares) prefetch_rows<F>(make_unit(&group, &chunk), lane);
  if (!grid_barrier(p.sync + 1, &r, p)) return;
  // h, 128 columns of a pair at a time: the parts of gate and of up joined, by a
  // CTA where there is one for each task, else by a warp
  {
    const int tiles = up_tiles, tasks = pairs * tiles, parts = up.chunks;
    auto parts_of = [&](int q, int tile, int half, int i, int n) {  // the i-th of n shares of the parts
      return add_parts(p.part1 + ((size_t)q * 2 + half) * p.f + tile * 128 + 4 * lane, up_slab, parts * i / n,
                       parts * (i + 1) / n);
    };
    const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
    if (tasks <= (int)gridDim.x) {
      const int q = blockIdx.x / tiles, tile = blockIdx.x % tiles;
      if (q < pairs) {
        const bool in = tile * 128 + 4 * lane < p.f;
        work.join[warp][lane] = in ? parts_of(q, tile, warp / 4, warp % 4, 4) : zero;
        __syncthreads();
        if (warp == 0) {
          float4 s[2];
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            s[half] = work.join[4 * half][lane];
#pragma unroll
            for (int i = 1; i < 4; ++i) s[half] = add4(s[half], work.join[4 * half + i][lane]);
          }
          put_h<F>(p, q, tile * 128 + 4 * lane, s[0], s[1], in);
        }
      }
    } else {
      for (int i = me; i < tasks; i += workers) {
        const int q = i / tiles, tile = i % tiles;
        const bool in = tile * 128 + 4 * lane < p.f;
        const float4 g = in ? parts_of(q, tile, 0, 0, 1) : zero, v = in ? parts_of(q, tile, 1, 0, 1) : zero;
        put_h<F>(p, q, tile * 128 + 4 * lane, g, v, in);
      }
    }
  }
  if (!grid_barrier(p.sync + 2, &r, p)) return;
  while (share < down.shares) {
    const unsigned next = ask_share(p.sync + kTaken2);
    const Unit u = make_unit(&group, &chunk);
    part_product<F, true>(p, &r, group, u, p.part2 + (size_t)chunk * down_slab, p.d, smem);
    share = down_taken + (int)__shfl_sync(0xffffffffu, next, 0);
  }
  if (!grid_barrier(p.sync + 3, &r, p)) return;

  // ------------------------------------------------------------------ y
  // 128 columns of a token by a CTA: `per` warps join the parts of an expert;
  // the experts' sums are added in their order
  {
    const int per = p.k > 4 ? 1 : p.k > 2 ? 2 : p.k == 2 ? 4 : 8, slots = kWarps / per;
    const int tiles = down_tiles, tasks = p.M * tiles, parts = down.chunks;
    for (int task = blockIdx.x; task < tasks; task += gridDim.x) {
      const int m = task / tiles, tile = task % tiles, c = tile * 128 + 4 * lane;
      float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int s0 = 0; s0 < p.k; s0 += slots) {
        const int s = s0 + warp / per;
        if (s < p.k && c < p.d) {
          const int q = m * p.k + s;
          work.join[warp][lane] = add_parts(p.part2 + (size_t)q * p.d + c, down_slab, parts * (warp % per) / per,
                                            parts * (warp % per + 1) / per);
        }
        __syncthreads();
        if (warp == 0 && c < p.d)
          for (int i = 0; i < slots && s0 + i < p.k; ++i) {
            float4 v = work.join[i * per][lane];
            for (int j = 1; j < per; ++j) v = add4(v, work.join[i * per + j][lane]);
            const float gate = r.gate[m * p.k + s0 + i];
            y = make_float4(fmaf(gate, v.x, y.x), fmaf(gate, v.y, y.y), fmaf(gate, v.z, y.z), fmaf(gate, v.w, y.w));
          }
        __syncthreads();
      }
      if (warp == 0 && c < p.d) *reinterpret_cast<float4*>(p.y + (size_t)m * p.d + c) = y;
    }
  }

  // the barriers' words are zero again once every CTA has passed the last one
  if (tid == 0 && atomic_add_acq_rel_gpu(p.sync + kSyncEnd, 1u) == gridDim.x - 1u) {
#pragma unroll
    for (int i = 0; i < kSyncWords; ++i) p.sync[i] = 0u;
  }
}

struct MoePlan {
  size_t logits, xop, hop, part1, part2, total;
};

MoePlan make_plan(int M, int d, int f, int E, int k, MoeFormat fmt) {
  MoePlan pl;
  const int rounds = fmt == MoeFormat::MX4 ? Cfg<Fmt::MX4>::kRounds : Cfg<Fmt::BF16>::kRounds;
  const int step = fmt == MoeFormat::BF16 ? 16 : fmt == MoeFormat::F32 ? 8 : 32;
  const int ctas = fmt == MoeFormat::MX4   ? Cfg<Fmt::MX4>::kCtas
                   : fmt == MoeFormat::F32 ? Cfg<Fmt::F32>::kCtas
                                           : Cfg<Fmt::BF16>::kCtas;
  const int workers = 148 * ctas * kWarps;
  // A unit has the most chunks where there are the fewest units: there are at
  // least k groups (a token's experts differ) and one for every eight pairs.
  const int groups = std::max(k, (M * k + kGroup - 1) / kGroup);
  const int parts1 = Cut::most(groups * 2 * ((f + 127) / 128), (d + step - 1) / step, workers, rounds);
  const int parts2 = Cut::most(groups * ((d + 127) / 128), (f + step - 1) / step, workers, rounds);
  const size_t pairs = (size_t)M * k;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off = (off + bytes + 255) / 256 * 256;
    return at;
  };
  pl.logits = take((size_t)M * E * 8);
  pl.xop = take(fmt == MoeFormat::MX4 ? (size_t)M * d * 4 + (size_t)M * (d / 32) * 4 : 0);
  pl.hop = take(pairs * f * (fmt == MoeFormat::BF16 ? 6 : 4) + pairs * (f / 32 + 1) * 4);
  pl.part1 = take((size_t)parts1 * pairs * 2 * f * 4);
  pl.part2 = take((size_t)parts2 * pairs * d * 4);
  pl.total = off;
  return pl;
}

template <Fmt F>
cudaError_t launch_fmt(const MParams& p, cudaStream_t stream) {
  static int grids[64] = {0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (grids[dev] == 0) {
    int sms = 0, per = 0;
    e = cudaFuncSetAttribute(moe_kernel<F>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Cfg<F>::kSmem);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(moe_kernel<F>, cudaFuncAttributePreferredSharedMemoryCarveout,
                               cudaSharedmemCarveoutMaxShared);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, moe_kernel<F>, kT, Cfg<F>::kSmem);
    if (e != cudaSuccess) return e;
    if (per < 1) return cudaErrorLaunchOutOfResources;
    // at most the grid that the workspace is laid out for
    grids[dev] = std::min(std::min(per, Cfg<F>::kCtas) * sms, Cfg<F>::kCtas * 148);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grids[dev], 1, 1);
  cfg.blockDim = dim3(kT, 1, 1);
  cfg.dynamicSmemBytes = Cfg<F>::kSmem;
  cfg.stream = stream;
  // every CTA must be resident at once: they wait on one another at the barriers
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeCooperative;
  attr[0].val.cooperative = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, moe_kernel<F>, p);
}

}  // namespace

size_t moe_buffer_bytes(int M, int d, int f, int E, int k) {
  size_t n = 0;
  for (MoeFormat fmt : {MoeFormat::BF16, MoeFormat::F32, MoeFormat::MX4})
    n = std::max(n, make_plan(M, d, f, E, k, fmt).total);
  return n;
}

cudaError_t launch_moe(const MoeArgs& a, cudaStream_t stream) {
  const MoePlan pl = make_plan(a.M, a.d, a.f, a.E, a.k, a.format);
  unsigned char* buf = static_cast<unsigned char*>(a.buf);
  MParams p{};
  p.x = a.x;
  p.wr = a.Wr;
  p.gu = static_cast<const uint8_t*>(a.W_gu);
  p.gus = static_cast<const uint8_t*>(a.S_gu);
  p.dn = static_cast<const uint8_t*>(a.W_d);
  p.dns = static_cast<const uint8_t*>(a.S_d);
  p.y = a.y;
  p.idx = a.idx;
  p.gate = a.gate;
  p.sync = a.sync;
  p.logits = reinterpret_cast<double*>(buf + pl.logits);
  p.xop = buf + pl.xop;
  p.hop = buf + pl.hop;
  p.part1 = reinterpret_cast<float*>(buf + pl.part1);
  p.part2 = reinterpret_cast<float*>(buf + pl.part2);
  p.M = a.M;
  p.d = a.d;
  p.f = a.f;
  p.E = a.E;
  p.k = a.k;
  p.renormalize = a.renormalize ? 1 : 0;
  p.x_f32 = a.x_elem == Elem::F32 ? 1 : 0;
  p.dev_status = a.dev_status;
  p.wait_ns = wait_limit_ns();
  switch (a.format) {
    case MoeFormat::BF16: return launch_fmt<Fmt::BF16>(p, stream);
    case MoeFormat::F32: return launch_fmt<Fmt::F32>(p, stream);
    default: return launch_fmt<Fmt::MX4>(p, stream);
  }
}

}  // namespace larosa
