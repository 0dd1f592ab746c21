// Sparse linear with a 4-bit weight (sm_100a), 1 to 16 tokens:
//
//   y[m][j] = sum_k val[m][k] W[idx[m][k]][j],   W row-major [d_in x d_out]
//   in MX4 with its blocks down the rows: W[i][j] = e2m1[i][j] 2^(b[i/32][j]-127)
//
// ("La RoSA" summary, 方法详解 / 技术框架: the K kept entries of the rotated
// activation times their rows of the counter-rotated weight; the 4-bit
// storage of that weight is not on the pages.)
//
// It is a stream of the kept rows (half a byte per entry, and the scales,
// 1/32 of a byte per entry of the whole weight), bound by HBM -- as long as
// the 4-bit entries can be decoded and multiplied as fast as they arrive,
// 43 entries per clock and SM at 6.5 TB/s.  Decoding to fp32 and one FMA per
// entry and token would take 2.5 + M issue slots per entry out of 128 per
// clock; so the products run as mma.sync.m16n8k16 on f16 operands with fp32
// accumulators (tcgen05 would need every decoded entry written to shared
// memory and read back, 4 bytes of traffic per half byte of weight):
//   * an e2m1 value is exact in f16, and cvt makes two of them at a time.  A
//     lane loads the same 16 columns of four rows; joining the low (or high)
//     halves of the bytes of two rows gives the pairs along the reduction
//     that the A operand wants, so no value is moved after its conversion;
//   * a token's 32 coefficients of a block are divided by a power of two that
//     puts the largest in [2^14, 2^15) and split into two f16 pieces of 11
//     bits, v = (p0 + 2^-11 p1) 2^(e - 14): what p0 leaves has up to 12 bits,
//     so |error| <= 2^-23 |v| for entries within 2^-27 of the block's largest
//     (below, 2^-50 of the largest); a third piece for the last bit would take
//     half as many MMAs again.  The pieces are neighbouring columns of the B
//     operand: 4 tokens x 2 pieces fill its 8 columns;
//   * a block's product is a fresh accumulator, scaled by the two powers of
//     two (the token's and the column's) when it is added to the fp32 sum.
//
// A warp takes a block of 32 rows by 128 columns (64-byte row segments).  Its
// rows arrive by asynchronous 16-byte copies in the warp's own ring of shared
// memory tiles, two or three blocks ahead: registers for more than one block in
// flight would halve the warps an SM holds.  Every copy is unconditional: an
// empty slot names a row of the block that is read anyway (its coefficient is
// zero), and columns past the matrix name the last ones (their sums are not
// written).  A CTA's warps take the blocks of one split in turn and add their
// sums in warp order through shared memory.  The splits of a column tile write
// their sums to the workspace, and the last one to arrive adds them in split
// order, so the result does not depend on timing.  (As thread-block clusters
// with distributed shared memory the splits left SMs empty: of clusters of
// seven, one CTA per SM, 15 fit the GPU at a time.)
//
// Two ways to the B operand, by the number of tokens:
//   up to 4 tokens   the CTA makes the operands of its split's blocks in
//                    shared memory from the tokens' fp32 coefficients (a kept
//                    list it scatters itself, or dense rows in global memory),
//                    both pieces of four tokens in one MMA's eight columns,
//                    and packs the rows some token keeps into steps of 16 and
//                    8 rows: at 60 % kept a block takes 24 of 32 slots.  One
//                    or two warps abreast (128 or 256 columns per CTA) share
//                    them;
//   5 to 16 tokens   the operand is made once, by eight CTAs per token or by the
//                    Top-K, and copied along with the rows: making it in every
//                    column tile would cost as much as the product (348 us
//                    where this takes 31).  An MMA holds one piece of eight
//                    tokens, so that a lane's neighbouring accumulators are two
//                    tokens and are scaled as pairs.  Nearly every row is kept
//                    by some token, so rows are not packed; one that no token
//                    keeps is replaced by one that is read anyway.
//
// Measured (B200, graph replay, weights from HBM): 2458 kept rows of 4096 x
// 22016, one token, 17.3 us for a given list (30 MB: 1.7 TB/s) and 22.4 with
// the Top-K before it (4 tokens 22.9 and 28.3, 8 tokens 25.2 and 30.9, 16 tokens
// 43.0 and 49.3); 8295 of 13824 x 5120, 16 tokens, 30.8 us with the operand kernel
// (39 MB: 1.3 TB/s).  One token is bound by the chain before the first block
// (scanning the list about 2.5 us, packing 1.5) and then by issue, about 250
// instructions a block; 16 tokens by no rate alone: 64 mma.sync a block at about 2.1
// clocks and SM are 8 us, its 550 instructions 9 us of issue, and three warps per
// scheduler do not cover one another's waits; the operand kernel before takes 8 us by
// itself, part of it beside the product's start.
#include <algorithm>

#include "common.cuh"
#include "internal.h"
#include "mx4.cuh"
#include "mx4_mma.cuh"

namespace larosa {
namespace {

constexpr int kRThreads = 256;
constexpr int kRWarps = kRThreads / 32;
constexpr int kFewRing = 3;   // up to 4 tokens
constexpr int kFewCtas = 3;   // CTAs per SM, up to 4 tokens
constexpr int kMaxSplits = 16;
constexpr int kMaxSplitRows = 16384;  // rows of one split a kept list is scattered into

struct RParams {
  const int32_t* idx;  // kept list (one token), or null
  const float* val;
  const float* coef;  // dense coefficient rows [M x d_in], or null
  mx4::Operand op;    // prepared operands (5 to 16 tokens)
  const uint8_t* codes;
  const uint8_t* scales;
  float* y;
  float* partials;    // [splits][tile][M][columns of a tile]
  unsigned* tickets;  // a word per tile, zero between calls
  int M, K, d_in, d_out;
  int blocks_per_split;
  int* dev_status;
};

// Adds the CTA's sums part[block lane][token][column] in lane order, then
// those of the tile's splits in split order, to y.
template <int kTok, int kHalves, int kThreads = kRThreads>
__device__ __forceinline__ void add_parts(float* part, const RParams& p) {
  constexpr int kCols = 128 * kHalves;
  __shared__ unsigned s_order;
  const int tid = threadIdx.x;
  __syncthreads();
  const int S = gridDim.x, tile = blockIdx.y, count = p.M * kCols;
  float* slab = p.partials + ((size_t)blockIdx.x * gridDim.y + tile) * count;
  for (int e = tid; e < count / 4; e += kThreads) {
    const float4* from = reinterpret_cast<const float4*>(part) + e;
    float4 s = *from;
#pragma unroll
    for (int w = 1; w < kThreads / 32 / kHalves; ++w) {
      const float4 v = from[w * kTok * kCols / 4];
      s.x += v.x;
      s.y += v.y;
      s.z += v.z;
      s.w += v.w;
    }
    if (S > 1) {
      __stcg(reinterpret_cast<float4*>(slab) + e, s);
    } else {
      const int m = 4 * e / kCols, j = tile * kCols + 4 * e % kCols;
      if (j < p.d_out) *reinterpret_cast<float4*>(p.y + (size_t)m * p.d_out + j) = s;
    }
  }
  if (S == 1) return;
  __syncthreads();
  if (tid == 0) s_order = atomic_add_acq_rel_gpu(&p.tickets[tile], 1u);
  __syncthreads();
  if (s_order != (unsigned)S - 1u) return;
  // four columns at a time, every split's in flight, added in split order
  const size_t step = (size_t)gridDim.y * count / 4;
  for (int e = tid; e < count / 4; e += kThreads) {
    const float4* from = reinterpret_cast<const float4*>(p.partials + (size_t)tile * count) + e;
    float4 v[kMaxSplits];
#pragma unroll
    for (int i = 0; i < kMaxSplits; ++i)
      v[i] = i < S ? __ldcg(from + (size_t)i * step) : make_float4(0.f, 0.f, 0.f, 0.f);
    float4 s = v[0];
#pragma unroll
    for (int i = 1; i < kMaxSplits; ++i) {
      s.x += v[i].x;
      s.y += v[i].y;
      s.z += v[i].z;
      s.w += v[i].w;
    }
    const int m = 4 * e / kCols, j = tile * kCols + 4 * e % kCols;
    // rows of y are multiples of 128 bytes, so a group of four is inside or outside
    if (j < p.d_out) *reinterpret_cast<float4*>(p.y + (size_t)m * p.d_out + j) = s;
  }
  if (tid == 0) p.tickets[tile] = 0u;  // every split has arrived
}

// Copies of a block's tile by one warp: `count` positions (a multiple of 8)
// of 64 bytes, four lanes each, and the scales.  row(p) is the byte offset of
// position p's row from `base` (with the lane's chunk of the row).
template <typename Row>
__device__ __forceinline__ void copy_tile(mx4::Tile& tile, const uint8_t* base, int count, const uint8_t* scales,
                                          int lane, Row row) {
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (8 * j < count) {
      const int pos = 8 * j + (lane >> 2);
      mx4::copy16_l2(&tile.row[pos][16 * (lane & 3)], base + row(pos));
    }
  if (lane < 8) mx4::copy16_l2(&tile.scale[16 * lane], scales);
}

// ---------------------------------------------------------------- up to 4 tokens

// A block's packed operand for up to kM tokens.
template <int kM>
struct __align__(16) Packed {
  __half piece[2][2 * kM][16];  // [step][2 token + piece][slot]
  uint32_t off[32];        // byte offset of each tile position's row from the block's first row
  float sx[4];
  int n;  // slots in use
  int pad[3];
};

// Tile position of a slot when n are in use: 16-row steps hold row 4 t + i of
// the step at 4 i + t, 8-row ones (the rest fits eight) row 2 t + i.
__device__ __forceinline__ int position_of(int slot, int n) {
  const int s = slot & 15;
  const bool eight = slot < 16 ? n <= 8 : n <= 24;
  if (!eight) return (slot & 16) + (s & 3) * 4 + (s >> 2);
  return (slot & 16) + (s < 8 ? (s & 1) * 4 + (s >> 1) : s);
}

template <int kM>
struct FewSmem {
  static constexpr size_t kRingBytes = sizeof(mx4::Tile) * kFewRing * kRWarps;
  static constexpr size_t kChunk = kM == 1 ? 48 : 32;  // blocks packed at a time
  static constexpr size_t kBytes = kRingBytes + kChunk * sizeof(Packed<kM>);
  static_assert((size_t)kRWarps * 4 * 128 * 4 <= kRingBytes, "the sums reuse the rings");
};

// kM: 1 for one token, 4 for two to four.
template <bool kList, int kM, int kHalves>
__global__ void __launch_bounds__(kRThreads, kFewCtas) mx4_rows_few_kernel(const RParams p) {
  constexpr int kLanes = kRWarps / kHalves;
  constexpr int kFewChunk = (int)FewSmem<kM>::kChunk;
  extern __shared__ __align__(16) unsigned char smem[];
  Packed<kM>* ops = reinterpret_cast<Packed<kM>*>(smem + FewSmem<kM>::kRingBytes);
  float* stage = reinterpret_cast<float*>(smem + FewSmem<kM>::kBytes);  // kList: the split's coefficients

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t = lane & 3;
  // this lane's column of the B operand; with one token only two exist, and
  // the others' products are never added
  const int gb = g % (2 * kM);
  mx4::Tile* ring = reinterpret_cast<mx4::Tile*>(smem) + warp * kFewRing;
  const int n_blocks = p.d_in / mx4::kBlock;
  const int b_begin = blockIdx.x * p.blocks_per_split;
  const int b_end = min(n_blocks, b_begin + p.blocks_per_split);
  const int col0 = (int)blockIdx.y * 128 * kHalves + (warp % kHalves) * 128;
  const uint32_t row_bytes = (uint32_t)p.d_out / 2;
  // this lane's copies: 16 bytes of rows and of scales, the last ones where
  // they lie past the matrix
  const uint32_t chunk = min((uint32_t)col0 / 2 + 16u * (lane & 3), row_bytes - 16u);
  const uint32_t s_col = (uint32_t)min(col0 + 16 * lane, p.d_out - 16);

  float acc[1][8][2];
#pragma unroll
  for (int q = 0; q < 8; ++q) acc[0][q][0] = acc[0][q][1] = 0.f;

  if constexpr (kList) {
    const int rows = max(b_end - b_begin, 0) * 32;
    for (int i = tid; i < rows / 4; i += kRThreads)
      reinterpret_cast<float4*>(stage)[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    __syncthreads();
    pdl_wait();
    pdl_launch_dependents();
    bool bad = false;
    const unsigned first = (unsigned)b_begin * 32u;
    constexpr int kBatch = 16;  // entries in flight per thread
    for (int i0 = tid; i0 < p.K; i0 += kBatch * kRThreads) {
      unsigned r[kBatch];
      float v[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int i = i0 + k * kRThreads;
        r[k] = i < p.K ? (unsigned)__ldg(p.idx + i) : first;
        v[k] = i < p.K ? __ldg(p.val + i) : 0.f;
      }
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        if (i0 + k * kRThreads >= p.K) break;
        if (r[k] - first < (unsigned)rows) stage[r[k] - first] = v[k];
        bad |= r[k] >= (unsigned)p.d_in;
      }
    }
    if (__any_sync(0xffffffffu, bad) && lane == 0) report(p.dev_status, LAROSA_DEV_INDEX);
  } else {
    pdl_wait();
    pdl_launch_dependents();
  }

  for (int c0 = b_begin; c0 < b_end; c0 += kFewChunk) {
    const int nb = min(kFewChunk, b_end - c0);
    __syncthreads();  // the list is staged; the chunk before is used up
    // all of a warp's coefficients are loaded before the first is used
    constexpr int kPer = kFewChunk / kRWarps;
    float vs[kPer][kM];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int b = warp + i * kRWarps;
#pragma unroll
      for (int m = 0; m < kM; ++m) {
        if constexpr (kList)
          vs[i][m] = b < nb ? stage[(c0 - b_begin + b) * 32 + lane] : 0.f;
        else
          vs[i][m] = b < nb && m < p.M ? __ldg(p.coef + (size_t)m * p.d_in + (c0 + b) * 32 + lane) : 0.f;
      }
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int b = warp + i * kRWarps;
      if (b >= nb) break;
      Packed<kM>& o = ops[b];
      const float(&v)[kM] = vs[i];
      bool any = false;
#pragma unroll
      for (int m = 0; m < kM; ++m) any |= v[m] != 0.f;  // a coefficient of zero adds nothing
      const unsigned kept = __ballot_sync(0xffffffffu, any);
      const unsigned below = (1u << lane) - 1u;
      const int n_kept = __popc(kept);
      const int slot = any ? __popc(kept & below) : n_kept + __popc(~kept & below);
#pragma unroll
      for (int m = 0; m < kM; ++m) {
        if (m < p.M) {
          const unsigned top = __reduce_max_sync(0xffffffffu, __float_as_uint(v[m]) & 0x7fffffffu);
          float up, down;
          mx4::piece_scale(top, &up, &down);
          __half p0, p1;
          mx4::split_pieces(v[m] * up, &p0, &p1);
          o.piece[slot >> 4][2 * m][slot & 15] = p0;
          o.piece[slot >> 4][2 * m + 1][slot & 15] = p1;
          if (lane == 0) o.sx[m] = down;
        }
      }
      o.off[position_of(slot, n_kept)] = (any ? (uint32_t)lane : kept ? (uint32_t)__ffs(kept) - 1u : 0u) * row_bytes;
      if (lane == 0) o.n = n_kept;
    }
    __syncthreads();

    int b = warp / kHalves;
    int at = b;  // the block the copies have come to, its rows and its scales
    uint32_t rows_at = (uint32_t)(c0 + b) * 32u * row_bytes + chunk;  // a weight has at most 2^30 bytes
    uint32_t scales_at = (uint32_t)(c0 + b) * (uint32_t)p.d_out + s_col;
    auto copy = [&](mx4::Tile& tile) {
      if (at < nb) {
        const Packed<kM>& o = ops[at];
        const int n = o.n;
        if (n > 0)
          copy_tile(tile, p.codes, (n + 7) & ~7, p.scales + scales_at, lane,
                    [&](int pos) { return rows_at + o.off[pos]; });
      }
      at += kLanes;
      rows_at += kLanes * 32u * row_bytes;
      scales_at += kLanes * (uint32_t)p.d_out;
      mx4::copies_commit();
    };
#pragma unroll
    for (int s = 0; s < kFewRing - 1; ++s) copy(ring[s]);
    int now = 0, fill = kFewRing - 1;
    for (; b < nb; b += kLanes) {
      __syncwarp();  // every lane has read the tile that is filled next
      copy(ring[fill]);
      fill = fill + 1 == kFewRing ? 0 : fill + 1;
      mx4::copies_wait<kFewRing - 1>();
      __syncwarp();  // the other lanes' copies too
      const mx4::Tile& tile = ring[now];
      now = now + 1 == kFewRing ? 0 : now + 1;
      const Packed<kM>& o = ops[b];
      const int n = o.n;
      if (n == 0) continue;
      const float sx[1] = {o.sx[kM == 1 ? 0 : t]};
      mx4::RowSet rs;
      uint2 bop[2][1];
      if (n <= 8) {
        rs.read<2, 0>(tile, g, t);
        bop[0][0] = make_uint2(*reinterpret_cast<const uint32_t*>(&o.piece[0][gb][2 * t]), 0u);
        mx4::block_product<1, 2, 0>(rs, bop, sx, acc);
        continue;
      }
      bop[0][0] = *reinterpret_cast<const uint2*>(&o.piece[0][gb][4 * t]);
      if (n <= 16) {
        rs.read<4, 0>(tile, g, t);
        mx4::block_product<1, 4, 0>(rs, bop, sx, acc);
      } else if (n <= 24) {
        rs.read<4, 2>(tile, g, t);
        bop[1][0] = make_uint2(*reinterpret_cast<const uint32_t*>(&o.piece[1][gb][2 * t]), 0u);
        mx4::block_product<1, 4, 2>(rs, bop, sx, acc);
      } else {
        rs.read<4, 4>(tile, g, t);
        bop[1][0] = *reinterpret_cast<const uint2*>(&o.piece[1][gb][4 * t]);
        mx4::block_product<1, 4, 4>(rs, bop, sx, acc);
      }
    }
    mx4::copies_wait<0>();
  }
  __syncthreads();
  // [block lane][token][column]; lanes of tokens that do not exist hold
  // whatever their columns held, and only tokens below M are added
  float* part = reinterpret_cast<float*>(smem);
  float* mine = part + ((size_t)(warp / kHalves) * 4 + t) * (128 * kHalves) + (warp % kHalves) * 128 + g * 16;
#pragma unroll
  for (int q = 0; q < 8; q += 2)
    *reinterpret_cast<float4*>(mine + 2 * q) =
        make_float4(acc[0][q][0], acc[0][q][1], acc[0][q + 1][0], acc[0][q + 1][1]);
  add_parts<4, kHalves>(part, p);
}

// ---------------------------------------------------------------- 5 to 16 tokens

// A tile and its block's operand and token scales, O octets of tokens.
template <int O>
struct __align__(16) ManyTile {
  mx4::Tile rows;
  __half piece[2][O][2][8][16];
  float sx[8 * O];
};

// Sixteen tokens' accumulators and operands take 168 registers: twelve warps
// in one CTA per SM (with sixteen warps of 128 registers they spill).
template <int O>
struct ManyCfg {
  static constexpr int kThreads = O == 1 ? 256 : 384;
  static constexpr int kCtas = O == 1 ? 2 : 1;  // per SM
  static constexpr int kRing = O == 1 ? 3 : 4;  // tiles of a warp's ring
  static constexpr int kWarps = kThreads / 32;
  static constexpr size_t kBytes = sizeof(ManyTile<O>) * kRing * kWarps;
  static_assert((size_t)(kWarps / 2) * 8 * O * 256 * 4 <= kBytes, "the sums reuse the rings");
};

template <int O>
__global__ void __launch_bounds__(ManyCfg<O>::kThreads, ManyCfg<O>::kCtas) mx4_rows_many_kernel(const RParams p) {
  extern __shared__ __align__(16) unsigned char smem[];
  constexpr int kTok = 8 * O, kRing = ManyCfg<O>::kRing;
  constexpr int kHalves = 2, kLanes = ManyCfg<O>::kWarps / kHalves;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t = lane & 3;
  ManyTile<O>* ring = reinterpret_cast<ManyTile<O>*>(smem) + warp * kRing;
  const int n_blocks = p.d_in / mx4::kBlock;
  const int b_begin = blockIdx.x * p.blocks_per_split;
  const int b_end = min(n_blocks, b_begin + p.blocks_per_split);
  const int col0 = (int)blockIdx.y * 128 * kHalves + (warp % kHalves) * 128;
  int b = b_begin + warp / kHalves;
  mx4::BlockCopies copies;
  copies.start(p.codes, p.scales, p.d_out, min(col0, p.d_out - 32), max(32, min(128, p.d_out - col0)), b, kLanes, lane);

  unsigned long long acc[O][16];
#pragma unroll
  for (int o = 0; o < O; ++o)
#pragma unroll
    for (int c = 0; c < 16; ++c) acc[o][c] = 0ull;

  pdl_wait();
  pdl_launch_dependents();

  // this lane's token's kept rows of block b; all tokens' together
  auto read_mask = [&](int b) -> unsigned {
    return b < b_end && lane < p.M ? __ldg(p.op.mask + (size_t)b * kTok + lane) : 0u;
  };
  auto any_token = [&](unsigned m) -> unsigned { return __reduce_or_sync(0xffffffffu, m); };
  int at = b;  // the block the copies have come to
  auto copy = [&](unsigned kept, ManyTile<O>& tile) {
    if (kept == ~0u) {
      copies.next(tile.rows, lane);
    } else if (at < b_end) {
      // rows that no token keeps are replaced by the first that one does
      mx4::BlockCopies some = copies;
      const uint32_t first = kept ? (uint32_t)__ffs(kept) - 1u : 0u;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t row = mx4::BlockCopies::row_of(8 * j + (lane >> 2));
        if (!((kept >> row) & 1u)) some.off[j] = first * ((uint32_t)p.d_out / 2);
      }
      if (kept != 0u) some.next(tile.rows, lane);
      copies.rows += copies.row_step;
      copies.scales += copies.scale_step;
    }
    if (kept != 0u) {
      const unsigned char* src = reinterpret_cast<const unsigned char*>(p.op.piece) + (size_t)at * (1024 * O) + 16 * lane;
      unsigned char* dst = reinterpret_cast<unsigned char*>(tile.piece) + 16 * lane;
#pragma unroll
      for (int i = 0; i < 2 * O; ++i) mx4::copy16_l1(dst + 512 * i, src + 512 * i);
      if (lane < 2 * O) mx4::copy16_l1(&tile.sx[4 * lane], p.op.sx + (size_t)at * kTok + 4 * lane);
    }
    at += kLanes;
    mx4::copies_commit();
  };

  // kept[s]: rows of the block in tile s of the ring, and of the one after;
  // masks are read two blocks before they are needed
  unsigned kept[kRing], raw[kRing];
#pragma unroll
  for (int s = 0; s < kRing; ++s) raw[s] = read_mask(b + s * kLanes);
  unsigned raw_next = read_mask(b + kRing * kLanes);
#pragma unroll
  for (int s = 0; s < kRing; ++s) kept[s] = any_token(raw[s]);
#pragma unroll
  for (int s = 0; s < kRing - 1; ++s) copy(kept[s], ring[s]);
  int now = 0, fill = kRing - 1;
  for (; b < b_end; b += kLanes) {
    __syncwarp();  // every lane has read the tile that is filled next
    copy(kept[kRing - 1], ring[fill]);
    const unsigned after = any_token(raw_next);
    raw_next = read_mask(b + (kRing + 1) * kLanes);
    mx4::copies_wait<kRing - 1>();
    __syncwarp();  // the other lanes' copies too
    if (kept[0] != 0u) {
      const ManyTile<O>& tile = ring[now];
      mx4::RowSet rs;
      rs.read<4, 4>(tile.rows, g, t);
      uint2 bop[2][O][2];
      unsigned long long sx[O];
#pragma unroll
      for (int o = 0; o < O; ++o) {
#pragma unroll
        for (int step = 0; step < 2; ++step)
#pragma unroll
          for (int piece = 0; piece < 2; ++piece)
            bop[step][o][piece] = *reinterpret_cast<const uint2*>(&tile.piece[step][o][piece][g][4 * t]);
        sx[o] = *reinterpret_cast<const unsigned long long*>(&tile.sx[8 * o + 2 * t]);
      }
      mx4::block_product8<O>(rs, bop, sx, acc);
    }
    now = now + 1 == kRing ? 0 : now + 1;
    fill = fill + 1 == kRing ? 0 : fill + 1;
#pragma unroll
    for (int s = 0; s < kRing - 1; ++s) kept[s] = kept[s + 1];
    kept[kRing - 1] = after;
  }
  mx4::copies_wait<0>();
  __syncthreads();
  // [block lane][token][column]
  float* part = reinterpret_cast<float*>(smem);
  constexpr int kCols = 128 * kHalves;
  float* mine = part + ((size_t)(warp / kHalves) * kTok + 2 * t) * kCols + (warp % kHalves) * 128 + g * 16;
#pragma unroll
  for (int o = 0; o < O; ++o)
#pragma unroll
    for (int c = 0; c < 16; c += 4) {
      const float2 v[4] = {mx4::unpack2(acc[o][c]), mx4::unpack2(acc[o][c + 1]), mx4::unpack2(acc[o][c + 2]),
                           mx4::unpack2(acc[o][c + 3])};
      float* to = mine + (size_t)8 * o * kCols + c;
      *reinterpret_cast<float4*>(to) = make_float4(v[0].x, v[1].x, v[2].x, v[3].x);
      *reinterpret_cast<float4*>(to + kCols) = make_float4(v[0].y, v[1].y, v[2].y, v[3].y);
    }
  add_parts<kTok, kHalves, ManyCfg<O>::kThreads>(part, p);
}

// ---------------------------------------------------------------- kept lists to dense rows or operands

constexpr int kPThreads = 1024;

// The CTAs of a token each scatter the entries of the kept list that fall
// into their range of rows into shared memory, then write the range as a
// dense fp32 row (coef) or as the token's operand.  (Four CTAs: 31.4 us for 16
// tokens of 13824 x 5120 with the product, eight 30.8.)
constexpr int kCoefParts = 8;

__global__ void __launch_bounds__(kPThreads, 1)
    mx4_coef_kernel(const int32_t* __restrict__ idx, const float* __restrict__ val, int K, int d, float* coef,
                    mx4::Operand op, int* dev_status) {
  extern __shared__ __align__(16) float row[];
  const int m = blockIdx.x;
  const int blocks = d / mx4::kBlock;
  const int b0 = blockIdx.y * blocks / kCoefParts, b1 = (blockIdx.y + 1) * blocks / kCoefParts;
  const unsigned first = (unsigned)b0 * 32u, rows = (unsigned)(b1 - b0) * 32u;
  for (unsigned i = threadIdx.x; i < rows; i += kPThreads) row[i] = 0.f;
  __syncthreads();
  pdl_wait();
  pdl_launch_dependents();
  bool bad = false;
  constexpr int kBatch = 8;  // entries in flight per thread
  for (int k0 = threadIdx.x; k0 < K; k0 += kBatch * kPThreads) {
    unsigned r[kBatch];
    float v[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int k = k0 + i * kPThreads;
      r[i] = k < K ? (unsigned)__ldg(idx + (size_t)m * K + k) : 0u;
      v[i] = k < K ? __ldg(val + (size_t)m * K + k) : 0.f;
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if (k0 + i * kPThreads >= K) break;
      if (r[i] - first < rows) row[r[i] - first] = v[i];
      bad |= r[i] >= (unsigned)d;
    }
  }
  if (__syncthreads_or(bad) && threadIdx.x == 0) report(dev_status, LAROSA_DEV_INDEX);
  if (coef != nullptr) {
    for (unsigned i = threadIdx.x; i < rows; i += kPThreads) coef[(size_t)m * d + first + i] = row[i];
  } else {
    const int lane = threadIdx.x & 31;
    for (int b = b0 + (threadIdx.x >> 5); b < b1; b += kPThreads / 32) op.put(b, m, row[(b - b0) * 32 + lane], lane);
  }
}

// CTAs per column tile: the count that ends the last CTA first when `slots`
// of them run at a time, at least one block per warp (`lanes` blocks at a
// time).
int pick_splits(int tiles, int n_blocks, int lanes, int slots) {
  int best = 1;
  double best_t = 1e30;
  for (int S = 1; S <= kMaxSplits; ++S) {
    if (S > 1 && n_blocks < S * lanes) break;
    const long long waves = ((long long)tiles * S + slots - 1) / slots;
    const int per_warp = ((n_blocks + S - 1) / S + lanes - 1) / lanes;
    const double t = (double)waves * (per_warp + 3.0);  // 3: the CTA's fixed work, in blocks
    if (t < best_t * 0.999) {
      best_t = t;
      best = S;
    }
  }
  return best;
}

// Raises a kernel's dynamic shared memory limit, once per device, and gives
// it all of the unified L1 / shared storage, so that several CTAs fit.
template <typename F>
cudaError_t allow_smem(F* fn, size_t bytes, int (&done)[64]) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!done[dev]) {
    e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(fn, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
    if (e != cudaSuccess) return e;
    done[dev] = 1;
  }
  return cudaSuccess;
}

// Whether a CTA takes 256 columns (two warps abreast): from 5 tokens on, and
// for fewer where that still gives every SM its CTAs.
bool wide_tiles(int M, int d_out) {
  return mx4_rows_take_operand(M) || (d_out + 255) / 256 * kMaxSplits >= kFewCtas * 148;
}

// The column tiles of a product and the splits of each, from the sizes alone:
// the launch and the size of the partial sums' buffer both go by it.
struct RowsPlan {
  int tiles, splits, blocks_per_split;
  int tile_cols;
};

RowsPlan rows_plan(int M, int d_in, int d_out, bool list) {
  const int halves = wide_tiles(M, d_out) ? 2 : 1;
  const int warps = M <= 8 ? kRWarps : ManyCfg<2>::kWarps;
  const int ctas = M <= 4 ? kFewCtas : M <= 8 ? ManyCfg<1>::kCtas : ManyCfg<2>::kCtas;
  const int n_blocks = d_in / mx4::kBlock;
  RowsPlan pl;
  pl.tile_cols = 128 * halves;
  pl.tiles = (d_out + pl.tile_cols - 1) / pl.tile_cols;
  pl.splits = pick_splits(pl.tiles, n_blocks, warps / halves, ctas * 148);
  if (list)  // the split's coefficients are staged in shared memory
    while (((n_blocks + pl.splits - 1) / pl.splits) * 32 > kMaxSplitRows) ++pl.splits;
  pl.blocks_per_split = (n_blocks + pl.splits - 1) / pl.splits;
  return pl;
}

template <typename F>
cudaError_t launch_tiles(F* fn, RParams p, int warps, size_t smem, cudaStream_t stream) {
  const RowsPlan pl = rows_plan(p.M, p.d_in, p.d_out, p.idx != nullptr);
  p.blocks_per_split = pl.blocks_per_split;
  if (p.idx != nullptr) smem += (size_t)pl.blocks_per_split * 32 * 4;
  const int S = pl.splits, tiles = pl.tiles;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(S, tiles, 1);
  cfg.blockDim = dim3(32 * warps, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fn, p);
}

template <bool kList, int kM, int kHalves>
cudaError_t launch_few(const RParams& p, cudaStream_t stream) {
  constexpr size_t kBytes = FewSmem<kM>::kBytes;
  static int done[64] = {0};
  auto* fn = mx4_rows_few_kernel<kList, kM, kHalves>;
  const cudaError_t e = allow_smem(fn, kBytes + (kList ? (size_t)kMaxSplitRows * 4 : 0), done);
  if (e != cudaSuccess) return e;
  return launch_tiles(fn, p, kRWarps, kBytes, stream);
}

template <bool kList, int kM>
cudaError_t launch_few(const RParams& p, cudaStream_t stream) {
  return wide_tiles(p.M, p.d_out) ? launch_few<kList, kM, 2>(p, stream) : launch_few<kList, kM, 1>(p, stream);
}

template <int O>
cudaError_t launch_many(const RParams& p, cudaStream_t stream) {
  using C = ManyCfg<O>;
  static int done[64] = {0};
  cudaError_t e = allow_smem(mx4_rows_many_kernel<O>, C::kBytes, done);
  if (e != cudaSuccess) return e;
  return launch_tiles(mx4_rows_many_kernel<O>, p, C::kWarps, C::kBytes, stream);
}

// Octets of tokens an operand is laid out for (1 to 4 tokens use none).
int octets_of(int M) { return (M + 7) / 8; }

mx4::Operand operand_at(void* buf, int M, int d_in) {
  mx4::Operand op;
  op.octets = octets_of(M);
  const size_t blocks = (size_t)d_in / mx4::kBlock;
  op.piece = static_cast<__half*>(buf);
  op.sx = reinterpret_cast<float*>(op.piece + blocks * 512 * op.octets);
  op.mask = reinterpret_cast<unsigned*>(op.sx + blocks * 8 * op.octets);
  return op;
}

}  // namespace

bool mx4_rows_take_operand(int M) { return M > 4; }

namespace {
// Bytes of the coefficients at the start of the buffer; the splits' partial
// sums follow.
size_t coef_bytes(int M, int d_in) {
  const size_t blocks = (size_t)d_in / mx4::kBlock;
  const size_t n = mx4_rows_take_operand(M) ? blocks * octets_of(M) * (1024 + 8 * 4 + 8 * 4) : (size_t)M * d_in * 4;
  return (n + 255) / 256 * 256;
}
}  // namespace

size_t mx4_rows_buffer_bytes(int M, int d_in, int d_out) {
  size_t partials = 0;  // of a single split: none
  for (bool list : {false, true}) {
    if (list && M != 1) break;  // only one token's list is read by the product
    const RowsPlan pl = rows_plan(M, d_in, d_out, list);
    if (pl.splits > 1) partials = std::max(partials, (size_t)pl.splits * pl.tiles * M * pl.tile_cols * 4);
  }
  return coef_bytes(M, d_in) + partials;
}

mx4::Operand mx4_rows_operand(void* buf, int M, int d_in) {
  return mx4_rows_take_operand(M) ? operand_at(buf, M, d_in) : mx4::Operand{};
}

cudaError_t launch_mx4_coef(const int32_t* idx, const float* val, int M, int K, int d_in, void* buf,
                            int* dev_status, cudaStream_t stream) {
  static int done[64] = {0};
  cudaError_t e = allow_smem(mx4_coef_kernel, (size_t)LAROSA_MAX_D * 4, done);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(M, kCoefParts, 1);
  cfg.blockDim = dim3(kPThreads, 1, 1);
  cfg.dynamicSmemBytes = (size_t)(d_in / mx4::kBlock + kCoefParts - 1) / kCoefParts * mx4::kBlock * 4;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const bool many = mx4_rows_take_operand(M);
  return cudaLaunchKernelEx(&cfg, mx4_coef_kernel, idx, val, K, d_in, many ? nullptr : static_cast<float*>(buf),
                            mx4_rows_operand(buf, M, d_in), dev_status);
}

cudaError_t launch_mx4_rows(const int32_t* idx, const float* val, int K, void* buf, unsigned* tickets, int M,
                            const void* codes, const void* scales, int d_in, int d_out, float* y, int* dev_status,
                            cudaStream_t stream) {
  RParams p{};
  p.codes = static_cast<const uint8_t*>(codes);
  p.scales = static_cast<const uint8_t*>(scales);
  p.y = y;
  p.partials = reinterpret_cast<float*>(static_cast<unsigned char*>(buf) + coef_bytes(M, d_in));
  p.tickets = tickets;
  p.M = M;
  p.K = K;
  p.d_in = d_in;
  p.d_out = d_out;
  p.dev_status = dev_status;
  if (!mx4_rows_take_operand(M)) {
    if (idx != nullptr && M != 1) return cudaErrorInvalidValue;
    p.idx = idx;
    p.val = val;
    p.coef = static_cast<const float*>(buf);
    if (idx != nullptr) return launch_few<true, 1>(p, stream);
    return M == 1 ? launch_few<false, 1>(p, stream) : launch_few<false, 4>(p, stream);
  }
  p.op = operand_at(buf, M, d_in);
  return M <= 8 ? launch_many<1>(p, stream) : launch_many<2>(p, stream);
}

}  // namespace larosa
