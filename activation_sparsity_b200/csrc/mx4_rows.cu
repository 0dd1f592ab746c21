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
//     bits, v = (p0 + 2^-11 p1) 2^(e - 14): |error| <= 2^-24 |v| for entries
//     within 2^-29 of the block's largest (below, 2^-50 of the largest).  The
//     pieces are neighbouring columns of the B operand: 4 tokens x 2 pieces
//     fill its 8 columns;
//   * a block's product is a fresh accumulator, scaled by the two powers of
//     two (the token's and the column's) when it is added to the fp32 sum.
//
// A warp takes a block of 32 rows by 128 columns (64-byte row segments: a
// lane's 16 columns are 8 bytes) and loads the next block while it multiplies
// this one.  A CTA's eight warps take the blocks of one split in turn and add
// their sums in warp order through shared memory; the splits of a column
// tile are a thread-block cluster whose CTAs add their tiles through
// distributed shared memory in rank order, so the result does not depend on
// timing.
//
// Two ways to the B operand, by the number of tokens:
//   up to 4 tokens   every warp makes the operand of its own block from the
//                    tokens' fp32 coefficients (a kept list scattered into
//                    shared memory by the CTA, or dense rows in global
//                    memory) and packs the rows some token keeps into as few
//                    16-row steps as they fill;
//   5 to 16 tokens   the operand is made once, by one CTA per token, and read
//                    through L1 by two warps side by side (256 columns per
//                    CTA): making it in every column tile would cost as much
//                    as the product.  Nearly every row is kept by some token,
//                    so rows are not packed, only left unread where no token
//                    keeps them.
#include <cooperative_groups.h>

#include <algorithm>

#include "common.cuh"
#include "internal.h"
#include "mx4.cuh"
#include "mx4_mma.cuh"

namespace cg = cooperative_groups;

namespace larosa {
namespace {

constexpr int kRThreads = 256;
constexpr int kRWarps = kRThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kMaxSplitRows = 16384;  // rows of one split a kept list is scattered into

struct RParams {
  const int32_t* idx;  // kept list (one token), or null
  const float* val;
  const float* coef;  // dense coefficient rows [M x d_in], or null
  mx4::Operand op;    // prepared operands (5 to 16 tokens)
  const uint8_t* codes;
  const uint8_t* scales;
  float* y;
  int M, K, d_in, d_out;
  int blocks_per_split;
  int* dev_status;
};

// The CTA's sums of every warp, added in warp order, then over the cluster in
// rank order, to y.  Warp w holds columns (w % kHalves) 128 ... of the tile.
template <int NT, int kHalves>
__device__ __forceinline__ void reduce_tile(const float (&acc)[NT][8][2], float* part, const RParams& p) {
  constexpr int kTok = 4 * NT;
  constexpr int kCols = 128 * kHalves;
  cg::cluster_group cluster = cg::this_cluster();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t = lane & 3;
  // [block lane][token][column]
  float* mine = part + ((size_t)(warp / kHalves) * kTok + t) * kCols + (warp % kHalves) * 128 + g * 16;
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int q = 0; q < 8; ++q)
      *reinterpret_cast<float2*>(mine + (size_t)4 * n * kCols + 2 * q) = make_float2(acc[n][q][0], acc[n][q][1]);
  __syncthreads();
  for (int e = tid; e < p.M * kCols; e += kRThreads) {
    float s = part[e];
#pragma unroll
    for (int w = 1; w < kRWarps / kHalves; ++w) s += part[w * kTok * kCols + e];
    part[e] = s;  // this thread's own element: no other reads it before the barrier
  }
  const int R = static_cast<int>(cluster.num_blocks());
  if (R > 1)
    cluster.sync();
  else
    __syncthreads();
  const int q0 = blockIdx.x * kCols / R, width = (blockIdx.x + 1) * kCols / R - q0;
  for (int e = tid; e < p.M * width; e += kRThreads) {
    const int m = e / width, c = q0 + e % width;
    const int j = blockIdx.y * kCols + c;
    float s = 0.f;
    for (int r = 0; r < R; ++r) s += cluster.map_shared_rank(part, r)[m * kCols + c];
    if (j < p.d_out) p.y[(size_t)m * p.d_out + j] = s;
  }
  if (R > 1) cluster.sync();  // no CTA leaves while another may still read its tile
}

// A warp's packed operand of one block, up to four tokens.
struct __align__(16) Packed {
  __half piece[2][8][16];  // [step][2 token + piece][slot]
  uint8_t row[32];         // row of each slot, 255 beyond the kept ones
  float sx[4];
};

// ---------------------------------------------------------------- up to 4 tokens

template <bool kList>
__global__ void __launch_bounds__(kRThreads, 2) mx4_rows_few_kernel(const RParams p) {
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ Packed s_op[kRWarps][2];
  float* stage = reinterpret_cast<float*>(smem);  // kList: the split's coefficients

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t = lane & 3;
  const int n_blocks = p.d_in / mx4::kBlock;
  const int b_begin = blockIdx.x * p.blocks_per_split;
  const int b_end = min(n_blocks, b_begin + p.blocks_per_split);
  const int col = blockIdx.y * 128 + g * 16;  // this lane's 16 columns
  const bool in = col < p.d_out;
  const size_t row_bytes = (size_t)p.d_out / 2;

  float acc[1][8][2];
#pragma unroll
  for (int q = 0; q < 8; ++q) acc[0][q][0] = acc[0][q][1] = 0.f;

  if constexpr (kList) {
    const int rows = (b_end - b_begin) * 32;
    for (int i = tid; i < rows / 4; i += kRThreads)
      reinterpret_cast<float4*>(stage)[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    __syncthreads();
    pdl_wait();
    pdl_launch_dependents();
    bool bad = false;
    for (int i = tid; i < p.K; i += kRThreads) {
      const unsigned r = (unsigned)__ldg(p.idx + i);
      const float v = __ldg(p.val + i);
      if (r - (unsigned)b_begin * 32u < (unsigned)max(rows, 0) && r < (unsigned)p.d_in)
        stage[r - b_begin * 32] = v;
      bad |= r >= (unsigned)p.d_in;
    }
    if (__any_sync(0xffffffffu, bad) && lane == 0) report(p.dev_status, LAROSA_DEV_INDEX);
    __syncthreads();
  } else {
    pdl_wait();
    pdl_launch_dependents();
  }

  // coefficient of row `lane` of block b for token m
  auto coef = [&](int b, int m) -> float {
    if constexpr (kList) return stage[(b - b_begin) * 32 + lane];
    return __ldg(p.coef + (size_t)m * p.d_in + b * 32 + lane);
  };
  constexpr int kM = kList ? 1 : 4;
  float v[kM];
  auto read_coef = [&](int b) {
#pragma unroll
    for (int m = 0; m < kM; ++m) v[m] = b < b_end && m < p.M ? coef(b, m) : 0.f;
  };
  // packs block b's coefficients (in v) into `o`; returns the kept count
  auto pack = [&](Packed& o) -> int {
    bool any = false;
#pragma unroll
    for (int m = 0; m < kM; ++m) any |= v[m] != 0.f;  // a coefficient of zero adds nothing
    const unsigned kept = __ballot_sync(0xffffffffu, any);
    const unsigned below = (1u << lane) - 1u;
    const int n_kept = __popc(kept);
    const int slot = any ? __popc(kept & below) : n_kept + __popc(~kept & below);
    __syncwarp();
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
    o.row[slot] = any ? (uint8_t)lane : (uint8_t)255;
    __syncwarp();
    return n_kept;
  };
  auto fetch = [&](int b, const Packed& o, int n_kept, mx4::RowSet& rs) {
    rs.load(p.codes + (size_t)b * 32 * row_bytes + (col >> 1), row_bytes, p.scales + (size_t)b * p.d_out + col,
            in && n_kept > 0, [&](int step, int i) {
              const uint32_t r = *reinterpret_cast<const uint32_t*>(&o.row[16 * step + 4 * t]);
              return in ? (r >> (8 * i)) & 255u : 255u;
            });
  };

  mx4::RowSet cur, next;
  int n_cur = 0, n_next = 0, buf = 0;
  int b = b_begin + warp;
  if (b < b_end) {
    read_coef(b);
    n_cur = pack(s_op[warp][0]);
    fetch(b, s_op[warp][0], n_cur, cur);
    read_coef(b + kRWarps);
  }
  for (; b < b_end; b += kRWarps) {
    if (b + kRWarps < b_end) {
      n_next = pack(s_op[warp][buf ^ 1]);
      fetch(b + kRWarps, s_op[warp][buf ^ 1], n_next, next);
      read_coef(b + 2 * kRWarps);
    }
    if (n_cur > 0) {
      const Packed& o = s_op[warp][buf];
      uint2 bop[2][1];
#pragma unroll
      for (int step = 0; step < 2; ++step) bop[step][0] = *reinterpret_cast<const uint2*>(&o.piece[step][g][4 * t]);
      const float sx[1] = {o.sx[t]};
      mx4::block_product<1>(cur, n_cur > 16, bop, sx, acc);
    }
    cur = next;
    n_cur = n_next;
    buf ^= 1;
  }
  __syncthreads();
  // lanes of tokens that do not exist hold whatever their columns held; only
  // tokens below M are added
  reduce_tile<1, 1>(acc, reinterpret_cast<float*>(smem), p);
}

// ---------------------------------------------------------------- 5 to 16 tokens

template <int NT>
__global__ void __launch_bounds__(kRThreads, NT == 2 ? 2 : 1) mx4_rows_many_kernel(const RParams p) {
  extern __shared__ __align__(16) unsigned char smem[];
  constexpr int kTok = 4 * NT;
  constexpr int kHalves = 2, kLanes = kRWarps / kHalves;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t = lane & 3;
  const int n_blocks = p.d_in / mx4::kBlock;
  const int b_begin = blockIdx.x * p.blocks_per_split;
  const int b_end = min(n_blocks, b_begin + p.blocks_per_split);
  const int col = blockIdx.y * 128 * kHalves + (warp % kHalves) * 128 + g * 16;
  const bool in = col < p.d_out;
  const size_t row_bytes = (size_t)p.d_out / 2;

  float acc[NT][8][2];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int q = 0; q < 8; ++q) acc[n][q][0] = acc[n][q][1] = 0.f;

  pdl_wait();
  pdl_launch_dependents();

  // rows of block b that some token keeps
  auto kept_rows = [&](int b) -> unsigned {
    const unsigned m = b < b_end && lane < p.M ? __ldg(p.op.mask + (size_t)b * kTok + lane) : 0u;
    return __reduce_or_sync(0xffffffffu, m);
  };
  auto fetch = [&](int b, unsigned kept, mx4::RowSet& rs) {
    const unsigned mine = in ? kept >> (4 * t) : 0u;
    rs.load(p.codes + (size_t)b * 32 * row_bytes + (col >> 1), row_bytes, p.scales + (size_t)b * p.d_out + col,
            in && kept != 0u, [&](int step, int i) {
              return (mine >> (16 * step + i)) & 1u ? (uint32_t)(16 * step + 4 * t + i) : 255u;
            });
  };

  mx4::RowSet cur, next;
  int b = b_begin + warp / kHalves;
  unsigned k_cur = kept_rows(b), k_next = kept_rows(b + kLanes);
  if (b < b_end) fetch(b, k_cur, cur);
  for (; b < b_end; b += kLanes) {
    if (b + kLanes < b_end) fetch(b + kLanes, k_next, next);
    const unsigned k_after = kept_rows(b + 2 * kLanes);
    if (k_cur != 0u) {
      uint2 bop[2][NT];
      float sx[NT];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int step = 0; step < 2; ++step)
          bop[step][n] = __ldg(reinterpret_cast<const uint2*>(p.op.piece) +
                               ((((size_t)b * 2 + step) * NT + n) * 8 + g) * 4 + t);
        sx[n] = __ldg(p.op.sx + (size_t)b * kTok + 4 * n + t);
      }
      mx4::block_product<NT>(cur, true, bop, sx, acc);
    }
    cur = next;
    k_cur = k_next;
    k_next = k_after;
  }
  __syncthreads();
  reduce_tile<NT, kHalves>(acc, reinterpret_cast<float*>(smem), p);
}

// ---------------------------------------------------------------- kept lists to dense rows or operands

constexpr int kPThreads = 1024;

// One CTA per token scatters the kept list into a row of shared memory, then
// writes it as a dense fp32 row (coef) or as the token's operand.
__global__ void __launch_bounds__(kPThreads, 1)
    mx4_coef_kernel(const int32_t* __restrict__ idx, const float* __restrict__ val, int K, int d, float* coef,
                    mx4::Operand op, int* dev_status) {
  extern __shared__ __align__(16) float row[];
  const int m = blockIdx.x;
  for (int i = threadIdx.x; i < d; i += kPThreads) row[i] = 0.f;
  __syncthreads();
  pdl_wait();
  pdl_launch_dependents();
  bool bad = false;
  for (int k = threadIdx.x; k < K; k += kPThreads) {
    const int i = __ldg(idx + (size_t)m * K + k);
    if (static_cast<unsigned>(i) < static_cast<unsigned>(d))
      row[i] = __ldg(val + (size_t)m * K + k);
    else
      bad = true;
  }
  if (__syncthreads_or(bad) && threadIdx.x == 0) report(dev_status, LAROSA_DEV_INDEX);
  if (coef != nullptr) {
    for (int i = threadIdx.x; i < d; i += kPThreads) coef[(size_t)m * d + i] = row[i];
  } else {
    const int lane = threadIdx.x & 31;
    for (int b = threadIdx.x >> 5; b < d / mx4::kBlock; b += kPThreads / 32) op.put(b, m, row[b * 32 + lane], lane);
  }
}

// CTAs per column tile: the count that ends the slowest CTA first when
// `slots` CTAs run at a time, at most eight (the portable cluster size) and
// at least one block per warp.
int pick_cluster(int tiles, int n_blocks, int lanes, int slots) {
  int best = 1;
  double best_t = 1e30;
  for (int S = 1; S <= kMaxCluster; S *= 2) {
    if (S > 1 && n_blocks < S * lanes) break;
    const double waves = std::max(1.0, (double)((long long)tiles * S) / slots);
    const int per_warp = ((n_blocks + S - 1) / S + lanes - 1) / lanes;
    const double t = waves * (per_warp + 3.0);  // 3: the CTA's fixed work, in blocks
    if (t < best_t * 0.999) {
      best_t = t;
      best = S;
    }
  }
  return best;
}

// Raises a kernel's dynamic shared memory limit, once per device.
template <typename F>
cudaError_t allow_smem(F* fn, size_t bytes, int (&done)[64]) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!done[dev]) {
    e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e != cudaSuccess) return e;
    done[dev] = 1;
  }
  return cudaSuccess;
}

template <typename F>
cudaError_t launch_tiles(F* fn, RParams p, int cols, int lanes, int slots, size_t smem, cudaStream_t stream) {
  const int tiles = (p.d_out + cols - 1) / cols;
  const int n_blocks = p.d_in / mx4::kBlock;
  int S = pick_cluster(tiles, n_blocks, lanes, slots);
  if (p.idx != nullptr) {  // the split's coefficients are staged in shared memory
    while (((n_blocks + S - 1) / S) * 32 > kMaxSplitRows) S *= 2;
    smem = std::max(smem, (size_t)((n_blocks + S - 1) / S) * 32 * 4);
  }
  p.blocks_per_split = (n_blocks + S - 1) / S;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(S, tiles, 1);
  cfg.blockDim = dim3(kRThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = S;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, fn, p);
}

// Token groups of four an operand is laid out for (1 to 4 tokens use none).
int groups_of(int M) { return M <= 8 ? 2 : 4; }

mx4::Operand operand_at(void* buf, int M, int d_in) {
  mx4::Operand op;
  op.nt = groups_of(M);
  const size_t blocks = (size_t)d_in / mx4::kBlock;
  op.piece = static_cast<__half*>(buf);
  op.sx = reinterpret_cast<float*>(op.piece + blocks * 256 * op.nt);
  op.mask = reinterpret_cast<unsigned*>(op.sx + blocks * 4 * op.nt);
  return op;
}

}  // namespace

bool mx4_rows_take_operand(int M) { return M > 4; }

size_t mx4_rows_buffer_bytes(int M, int d_in) {
  if (!mx4_rows_take_operand(M)) return (size_t)M * d_in * 4;
  const size_t blocks = (size_t)d_in / mx4::kBlock;
  return blocks * groups_of(M) * (512 + 4 * 4 + 4 * 4);
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
  cfg.gridDim = dim3(M, 1, 1);
  cfg.blockDim = dim3(kPThreads, 1, 1);
  cfg.dynamicSmemBytes = (size_t)d_in * 4;
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

cudaError_t launch_mx4_rows(const int32_t* idx, const float* val, int K, const void* buf, int M, const void* codes,
                            const void* scales, int d_in, int d_out, float* y, int* dev_status,
                            cudaStream_t stream) {
  RParams p{};
  p.codes = static_cast<const uint8_t*>(codes);
  p.scales = static_cast<const uint8_t*>(scales);
  p.y = y;
  p.M = M;
  p.K = K;
  p.d_in = d_in;
  p.d_out = d_out;
  p.dev_status = dev_status;
  constexpr size_t kFewSmem = (size_t)kRWarps * 4 * 128 * 4;
  if (idx != nullptr) {
    if (M != 1) return cudaErrorInvalidValue;
    p.idx = idx;
    p.val = val;
    static int done[64] = {0};
    cudaError_t e = allow_smem(mx4_rows_few_kernel<true>, (size_t)kMaxSplitRows * 4, done);
    if (e != cudaSuccess) return e;
    return launch_tiles(mx4_rows_few_kernel<true>, p, 128, kRWarps, 2 * 148, kFewSmem, stream);
  }
  if (!mx4_rows_take_operand(M)) {
    p.coef = static_cast<const float*>(buf);
    return launch_tiles(mx4_rows_few_kernel<false>, p, 128, kRWarps, 2 * 148, kFewSmem, stream);
  }
  p.op = operand_at(const_cast<void*>(buf), M, d_in);
  constexpr size_t kManySmem = (size_t)(kRWarps / 2) * 4 * 256 * 4;  // per token group of four
  if (M <= 8) {
    static int done[64] = {0};
    cudaError_t e = allow_smem(mx4_rows_many_kernel<2>, 2 * kManySmem, done);
    if (e != cudaSuccess) return e;
    return launch_tiles(mx4_rows_many_kernel<2>, p, 256, kRWarps / 2, 2 * 148, 2 * kManySmem, stream);
  }
  static int done[64] = {0};
  cudaError_t e = allow_smem(mx4_rows_many_kernel<4>, 4 * kManySmem, done);
  if (e != cudaSuccess) return e;
  return launch_tiles(mx4_rows_many_kernel<4>, p, 256, kRWarps / 2, 148, 4 * kManySmem, stream);
}

}  // namespace larosa
