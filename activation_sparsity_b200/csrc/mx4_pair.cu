// Product of two MX4 matrices for many tokens: the same sums as
// mx4_linear.cu, on pairs of SMs (sm_100a, tcgen05 cta_group::2).
//
// With one SM per MMA tile, 128 outputs x 256 tokens, the codes reach the SMs
// too slowly: 48 KB per stage of 256 inputs and SM, of which the tensor core
// makes short work (4096 tokens of 5120 x 27648: 10.7 TB/s out of L2, 335 us of
// copies against about 130 us of MMAs).  A pair of CTAs shares one tile of 256
// outputs x NT tokens instead: each brings 128 rows of the weight and half of
// the tokens, 32 KB per stage at NT = 256, and the MMA of the pair reads both
// halves of the tokens.  Each CTA's TMEM holds the accumulators of its 128
// outputs for all NT tokens, the scales of its own rows and of every token.
//
// The scale bytes are first put in the order the tensor core reads them in
// (arrange_kernel: 512 bytes for 128 rows x 4 blocks, row r at 16 (r % 32) +
// 4 (r / 32)), in the workspace: 1/17 of the operands, one pass.  Gathered row
// by row inside the product, eight bytes of a 32-byte sector at a time, they
// cost more than the codes (230 of 640 us).
//
// The grid is persistent, a pair per two SMs; tokens vary fastest over the
// tiles, so the pairs at work share a few weight tiles and x stays in L2.
// Roles of a CTA's six warps:
//   0-3   epilogue: accumulators to shared memory in the output's type, then
//         256-byte rows to y, while the next tile is multiplied;
//   4     one thread: codes and scales by TMA, into this CTA's ring; both
//         CTAs' copies complete on the first CTA's `full` barriers;
//   5     one thread of the first CTA: scales to TMEM and MMAs for the pair;
//         tcgen05.commit returns a stage, or hands over a tile, in both CTAs.
// Every wait is bounded; a CTA that gives up reports and leaves its loops, and
// the pair leaves together.
#include <cooperative_groups.h>
#include <cuda.h>

#include <algorithm>

#include "common.cuh"
#include "internal.h"
#include "mx4_umma.cuh"

namespace cg = cooperative_groups;

namespace larosa {
namespace {

constexpr int kPThreads = 192;
using mx4::kStageK;

template <int NT>
struct PCfg {
  static constexpr int kHalves = (NT + 127) / 128;
  static constexpr int kStages = NT == 256 ? 4 : NT == 192 ? 5 : 6;
  static constexpr uint32_t kA = 128 * 128, kB = NT / 2 * 128;
  static constexpr uint32_t kSfA = 1024, kSfB = 1024 * kHalves;
  static constexpr uint32_t kStage = kA + kB + kSfA + kSfB;
  static constexpr uint32_t kOut = NT * 128 * 2;  // NT tokens in bf16, half of them in fp32
  static constexpr int kSfCols = 8 + 8 * kHalves;
  static constexpr int kTmemCols = 512;
  static constexpr size_t kSmem = (size_t)kStages * kStage + kOut + 1024;
  static_assert(kStage % 1024 == 0, "swizzled stages stay 1024-byte aligned");
  static_assert(NT + kStages * kSfCols <= kTmemCols, "TMEM");
  static_assert(kSmem <= 227 * 1024, "shared memory");
};

struct PParams {
  void* y;
  int out_bf16;
  int M, d_in, d_out;
  int tn, tiles;  // token tiles, all tiles
  int* dev_status;
  unsigned long long wait_ns;
};

// Address of this CTA's shared variable in the first CTA of the pair.
__device__ __forceinline__ uint32_t in_first(const void* p) {
  uint32_t a;
  asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(a) : "r"(smem_u32(p)));
  return a;
}

__device__ __forceinline__ void arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// mbar_wait_bounded for a barrier that the other CTA of the pair arrives at.
__device__ __forceinline__ bool wait_cluster(uint64_t* bar, uint32_t parity, volatile int* abort,
                                             unsigned long long limit_ns) {
  unsigned long long t0 = 0;
  for (uint32_t it = 0;; ++it) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    if (done) return true;
    if ((it & 255u) == 255u) {
      if (*abort) return false;
      const unsigned long long now = global_timer_ns();
      if (t0 == 0) t0 = now;
      if (now - t0 > limit_ns) return false;
    }
  }
}

// TMA tile to this CTA's shared memory, completing on a barrier of the pair.
__device__ __forceinline__ void tma_load_pair(void* dst, const CUtensorMap* map, int c0, int c1, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
      " [%0], [%1, {%3, %4}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1)
      : "memory");
}

// Arrives at `bar` in both CTAs once every MMA issued so far has completed.
__device__ __forceinline__ void commit_pair(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
          smem_u32(bar)),
      "h"((uint16_t)3)
      : "memory");
}

// Whether any of the 128 threads of warps 0-3 passes true (barrier 1).
__device__ __forceinline__ bool any_of_128(bool mine) {
  int r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.s32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, 1, 128, p;\n\t"
      "selp.s32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((int)mine)
      : "memory");
  return r != 0;
}

template <int NT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPThreads, 1)
    mx4_pair_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x,
                    const __grid_constant__ CUtensorMap map_ws, const __grid_constant__ CUtensorMap map_xs,
                    const PParams p) {
  using C = PCfg<NT>;
  constexpr int kS = C::kStages;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* stages = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  unsigned char* out = stages + (size_t)kS * C::kStage;
  __shared__ uint64_t full[kS], empty[kS], acc_full, acc_empty;
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;

  cg::cluster_group cluster = cg::this_cluster();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = static_cast<int>(cluster.block_rank());
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  const int n_it = (p.d_in + kStageK - 1) / kStageK;

  if (tid == 0) {
    for (int s = 0; s < kS; ++s) {
      mbar_init(&full[s], 1);  // the first CTA's TMA thread, and the bytes of both
      mbar_init(&empty[s], 1);
    }
    mbar_init(&acc_full, 1);
    mbar_init(&acc_empty, 8);  // both CTAs' epilogue warps
    s_abort = 0;
    mbar_init_fence();
  }
  if (warp == 5) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s_tmem)),
                 "r"(C::kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc::tmem_fence_before();
  cluster.sync();  // the barriers of both CTAs are ready
  tc::tmem_fence_after();
  const uint32_t tmem = s_tmem;
  volatile int* abort_flag = &s_abort;

  pdl_wait();
  pdl_launch_dependents();

  if (warp < 4) {
    // ---------------------------------------------------------------- epilogue
    const int round_tokens = p.out_bf16 ? NT : NT / 2;  // tokens the staging area holds
    const size_t elem = p.out_bf16 ? 2 : 4;
    const uint32_t lanes = tmem + ((uint32_t)(warp * 32) << 16);
    int round = 0;
    bool ok = true;  // the same in all four warps
    for (int tile = pair; tile < p.tiles && ok; tile += pairs, ++round) {
      const int n0 = tile % p.tn * NT, j0 = tile / p.tn * 256 + rank * 128;
      ok = wait_cluster(&acc_full, round & 1, abort_flag, p.wait_ns);
      ok = !any_of_128(!ok);
      if (!ok) {
        *abort_flag = 1;
        break;
      }
      tc::tmem_fence_after();
      const int rows = min(128, p.d_out - j0);  // may be negative: nothing to write
      const bool wide = rows == 128 && ((size_t)p.d_out * elem) % 16 == 0;
      for (int t0 = 0; t0 < NT; t0 += round_tokens) {
        // the staging area is free: every warp has written its part of the round before
        asm volatile("bar.sync 1, 128;" ::: "memory");
#pragma unroll 1
        for (int c0 = 0; c0 < round_tokens; c0 += 32) {
          float v[32];
          tc::tmem_ld32(lanes + t0 + c0, v);
          if (p.out_bf16) {
            __nv_bfloat16* at = reinterpret_cast<__nv_bfloat16*>(out) + (size_t)c0 * 128 + tid;
#pragma unroll
            for (int c = 0; c < 32; ++c) at[c * 128] = __float2bfloat16_rn(v[c]);  // the caller's output type
          } else {
            float* at = reinterpret_cast<float*>(out) + (size_t)c0 * 128 + tid;
#pragma unroll
            for (int c = 0; c < 32; ++c) at[c * 128] = v[c];
          }
        }
        if (t0 + round_tokens >= NT) {  // the accumulators are read: the next tile may start
          tc::tmem_fence_before();
          __syncwarp();
          if (lane == 0) arrive_cluster(in_first(&acc_empty));
        }
        asm volatile("bar.sync 1, 128;" ::: "memory");
        const int tokens = min(round_tokens, p.M - n0 - t0);
        unsigned char* y = static_cast<unsigned char*>(p.y) + ((size_t)(n0 + t0) * p.d_out + j0) * elem;
        const size_t pitch = (size_t)p.d_out * elem;
        if (wide) {
          const int per_row = (int)(128 * elem / 16);  // 16-byte pieces of a token's outputs
          for (int i = tid; i < tokens * per_row; i += 128) {
            const int m = i / per_row, c = i % per_row;
            __stcs(reinterpret_cast<uint4*>(y + m * pitch + 16 * c),
                   *reinterpret_cast<const uint4*>(out + (size_t)m * 128 * elem + 16 * c));
          }
        } else if (tid < rows) {
          for (int m = 0; m < tokens; ++m) {
            if (p.out_bf16)
              reinterpret_cast<__nv_bfloat16*>(y + m * pitch)[tid] =
                  reinterpret_cast<const __nv_bfloat16*>(out)[(size_t)m * 128 + tid];
            else
              reinterpret_cast<float*>(y + m * pitch)[tid] = reinterpret_cast<const float*>(out)[(size_t)m * 128 + tid];
          }
        }
      }
    }
  } else if (warp == 4) {
    // ---------------------------------------------------------------- copies
    if (lane == 0) {
      long long g = 0;
      bool ok = true;
      for (int tile = pair; tile < p.tiles && ok; tile += pairs) {
        const int n0 = tile % p.tn * NT, j0 = tile / p.tn * 256;
        for (int it = 0; it < n_it; ++it, ++g) {
          const int s = (int)(g % kS);
          if (g >= kS && !wait_cluster(&empty[s], (uint32_t)((g / kS) - 1) & 1u, abort_flag, p.wait_ns)) {
            *abort_flag = 1;
            ok = false;
            break;
          }
          unsigned char* dst = stages + (size_t)s * C::kStage;
          if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * C::kStage);  // both CTAs' copies
          const uint32_t bar = in_first(&full[s]);
          tma_load_pair(dst, &map_w, it * 128, j0 + rank * 128, bar);
          tma_load_pair(dst + C::kA, &map_x, it * 128, n0 + rank * (NT / 2), bar);
          tma_load_pair(dst + C::kA + C::kB, &map_ws, 0, (j0 / 128 + rank) * n_it + it, bar);
          tma_load_pair(dst + C::kA + C::kB + C::kSfA, &map_xs, 0, (tile % p.tn * n_it + it) * C::kHalves, bar);
        }
      }
    }
  } else if (rank == 0) {
    // ---------------------------------------------------------------- MMA issuer
    if (lane == 0) {
      long long g = 0;
      int round = 0;
      bool ok = true;
      for (int tile = pair; tile < p.tiles && ok; tile += pairs, ++round) {
        if (round > 0 && !wait_cluster(&acc_empty, (uint32_t)(round - 1) & 1u, abort_flag, p.wait_ns)) {
          *abort_flag = 1;
          break;
        }
        tc::tmem_fence_after();
        for (int it = 0; it < n_it; ++it, ++g) {
          const int s = (int)(g % kS);
          if (!wait_cluster(&full[s], (uint32_t)(g / kS) & 1u, abort_flag, p.wait_ns)) {
            *abort_flag = 1;
            ok = false;
            break;
          }
          tc::tmem_fence_after();
          const uint32_t a_addr = smem_u32(stages + (size_t)s * C::kStage);
          const uint32_t b_addr = a_addr + C::kA, sfa = b_addr + C::kB, sfb = sfa + C::kSfA;
          const uint32_t ta = tmem + NT + s * C::kSfCols, tb = ta + 8;
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            mx4::copy_scales<2>(ta + 4 * c, sfa + 512 * c);
#pragma unroll
            for (int h = 0; h < C::kHalves; ++h)
              mx4::copy_scales<2>(tb + 4 * (c * C::kHalves + h), sfb + 512 * (c * C::kHalves + h));
          }
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)  // 64 inputs (32 bytes) each
            mx4::umma_mxf4<2>(tmem, tc::sw128_desc(a_addr + kk * 32), tc::sw128_desc(b_addr + kk * 32),
                              mx4::idesc_mxf4(256, NT, 2 * (kk & 1)), ta + 4 * (kk >> 1),
                              tb + 4 * C::kHalves * (kk >> 1), (it > 0 || kk > 0) ? 1u : 0u);
          commit_pair(&empty[s]);
        }
        if (ok) commit_pair(&acc_full);
      }
    }
  }
  __syncwarp();

  // ------------------------------------------------------------------ exit
  tc::tmem_fence_before();
  __syncthreads();
  if (tid == 0 && *abort_flag) report(p.dev_status, LAROSA_DEV_TIMEOUT);
  // no CTA leaves while the other may still arrive at its barriers or read
  // its shared memory
  cluster.sync();
  if (warp == 5) {
    tc::tmem_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(C::kTmemCols) : "memory");
  }
  cluster.sync();
}

// Scale bytes of a row-major [rows x blocks] matrix in the tensor core's order:
// per tile of `tile_rows` rows and stage of 8 blocks, two chunks of 4 blocks,
// each `halves` runs of 512 bytes (128 rows).  A thread takes four rows 32
// apart and four stages: 32 bytes of each row in, eight 16-byte words out.
// Rows and blocks past the matrix become zeros.
constexpr int kArrangeStages = 4;
constexpr int kArrangeThreads = 128;  // 32 row quads x 4 groups of stages

struct ArrangeParams {
  const uint8_t* src;
  uint4* dst;
  int rows, blocks, n_it;
  int tile_rows, halves;
  int row_runs;  // 128-row runs of all tiles
};

__device__ __forceinline__ void arrange(const ArrangeParams& p, int run, int it0) {
  const int r0 = threadIdx.x & 31;
  const int tile = run / p.halves, half = run % p.halves;
  uint32_t w[4][2 * kArrangeStages];  // [row][4 blocks]
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int in_tile = 128 * half + 32 * q + r0;
    const long long row = (long long)tile * p.tile_rows + in_tile;
    const bool in = in_tile < p.tile_rows && row < p.rows;
    const uint8_t* at = in ? p.src + row * p.blocks : nullptr;
#pragma unroll
    for (int s = 0; s < kArrangeStages; ++s) {
      const uint2 v = mx4::load_scales(at, p.blocks, (it0 + s) * mx4::kStageBlocks);
      w[q][2 * s] = v.x;
      w[q][2 * s + 1] = v.y;
    }
  }
#pragma unroll
  for (int s = 0; s < kArrangeStages; ++s) {
    if (it0 + s >= p.n_it) break;
#pragma unroll
    for (int c = 0; c < 2; ++c)
      p.dst[((((size_t)tile * p.n_it + it0 + s) * 2 + c) * p.halves + half) * 32 + r0] =
          make_uint4(w[0][2 * s + c], w[1][2 * s + c], w[2][2 * s + c], w[3][2 * s + c]);
  }
}

// The weight's scales, then x's.
__global__ void __launch_bounds__(kArrangeThreads) arrange_kernel(const ArrangeParams w, const ArrangeParams x) {
  pdl_wait();
  pdl_launch_dependents();
  const int it0 = (blockIdx.y * (kArrangeThreads / 32) + (threadIdx.x >> 5)) * kArrangeStages;
  if (it0 >= w.n_it) return;
  if ((int)blockIdx.x < w.row_runs)
    arrange(w, blockIdx.x, it0);
  else
    arrange(x, blockIdx.x - w.row_runs, it0);
}

// A tensor map of arranged scales: rows of 1024 bytes, `box_rows` at a time.
bool make_scale_map(CUtensorMap* map, const void* base, long long rows, int box_rows) {
  const tc::EncodeTiled enc = tc::encoder();
  if (enc == nullptr) return false;
  const cuuint64_t dims[2] = {256, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {1024};
  const cuuint32_t box[2] = {256, (cuuint32_t)box_rows};
  const cuuint32_t estr[2] = {1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, const_cast<void*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_NONE,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Pairs' weight tiles are 256 rows: two runs of 128, the second perhaps past
// the matrix.
long long weight_runs(int d_out) { return 2LL * ((d_out + 255) / 256); }

template <int NT>
cudaError_t launch_pair_nt(const void* xc, const void* xs, const void* wc, const void* ws, void* buf, PParams p,
                           cudaStream_t stream) {
  using C = PCfg<NT>;
  static int configured[64] = {0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!configured[dev]) {
    e = cudaFuncSetAttribute(mx4_pair_kernel<NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::kSmem);
    if (e != cudaSuccess) return e;
    configured[dev] = 1;
  }
  p.tn = (p.M + NT - 1) / NT;
  p.tiles = p.tn * ((p.d_out + 255) / 256);
  const int n_it = (p.d_in + kStageK - 1) / kStageK;
  const long long w_rows = weight_runs(p.d_out) * n_it, x_rows = (long long)p.tn * n_it * C::kHalves;
  unsigned char* wbuf = static_cast<unsigned char*>(buf);
  unsigned char* xbuf = wbuf + w_rows * 1024;
  CUtensorMap map_w, map_x, map_ws, map_xs;
  if (!mx4::make_byte_map(&map_w, wc, p.d_out, p.d_in / 2, 128) ||
      !mx4::make_byte_map(&map_x, xc, p.M, p.d_in / 2, NT / 2) || !make_scale_map(&map_ws, wbuf, w_rows, 1) ||
      !make_scale_map(&map_xs, xbuf, x_rows, C::kHalves))
    return cudaErrorInvalidValue;
  const int blocks = p.d_in / mx4::kBlock;
  const ArrangeParams aw{static_cast<const uint8_t*>(ws), reinterpret_cast<uint4*>(wbuf), p.d_out, blocks, n_it, 128, 1,
                         (int)weight_runs(p.d_out)};
  const ArrangeParams ax{static_cast<const uint8_t*>(xs), reinterpret_cast<uint4*>(xbuf), p.M, blocks, n_it, NT,
                         C::kHalves, p.tn * C::kHalves};
  cudaLaunchConfig_t cfg = {};
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  constexpr int kPerCta = kArrangeStages * kArrangeThreads / 32;
  cfg.gridDim = dim3(aw.row_runs + ax.row_runs, (n_it + kPerCta - 1) / kPerCta, 1);
  cfg.blockDim = dim3(kArrangeThreads, 1, 1);
  e = cudaLaunchKernelEx(&cfg, arrange_kernel, aw, ax);
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3(2 * std::min(74, p.tiles), 1, 1);
  cfg.blockDim = dim3(kPThreads, 1, 1);
  cfg.dynamicSmemBytes = C::kSmem;
  return cudaLaunchKernelEx(&cfg, mx4_pair_kernel<NT>, map_w, map_x, map_ws, map_xs, p);
}

}  // namespace

// Clocks of a shape with NT tokens per tile: rounds of the pairs times a
// tile's stages, each as long as its copies at 42 bytes per clock and SM (what
// L2 gives when every SM asks, measured) or its MMAs, and a fixed part.
double mx4_pair_clocks(int nt, int M, int d_in, int d_out) {
  const long long tiles = (long long)((M + nt - 1) / nt) * ((d_out + 255) / 256);
  const int n_it = (d_in + kStageK - 1) / kStageK;
  const double stage = std::max(2.0 * nt, (19456.0 + 64.0 * nt) / 42.0);
  return (double)((tiles + 73) / 74) * (n_it * stage + 1200.0) + 5000.0;
}

size_t mx4_pair_buffer_bytes(int M, int d_in, int d_out) {
  const long long n_it = (d_in + kStageK - 1) / kStageK;
  // x's tiles: of 128, 192 (two runs each) or 256 tokens (two runs)
  const long long x_runs = std::max((M + 127LL) / 128, std::max((M + 191LL) / 192 * 2, (M + 255LL) / 256 * 2));
  return (size_t)((weight_runs(d_out) + x_runs) * n_it * 1024);
}

cudaError_t launch_mx4_pair(int nt, const void* x_codes, const void* x_scales, const void* w_codes,
                            const void* w_scales, int M, int d_in, int d_out, void* y, bool out_bf16, void* buf,
                            int* dev_status, cudaStream_t stream) {
  PParams p{y, out_bf16 ? 1 : 0, M, d_in, d_out, 0, 0, dev_status, wait_limit_ns()};
  switch (nt) {
    case 128: return launch_pair_nt<128>(x_codes, x_scales, w_codes, w_scales, buf, p, stream);
    case 192: return launch_pair_nt<192>(x_codes, x_scales, w_codes, w_scales, buf, p, stream);
    default: return launch_pair_nt<256>(x_codes, x_scales, w_codes, w_scales, buf, p, stream);
  }
}

}  // namespace larosa
