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
// The scale bytes are first put in the order TMEM holds them in
// (arrange_kernel: 512 bytes for 128 rows x 4 blocks, row r at 16 (r % 32) +
// 4 (r / 32)), in the workspace: 1/17 of the operands, one pass.  Gathered row
// by row inside the product, eight bytes of a 32-byte sector at a time, they
// cost more than the codes (230 of 640 us).  Four warps load them into
// registers and store them to TMEM themselves: copied by the tensor core's own
// path (tcgen05.cp) they hold up the MMAs, six copies a stage at about 50
// clocks next to 512 clocks of MMAs (80 of 330 us).
//
// The grid is persistent, a pair per two SMs; tokens vary fastest over the
// tiles, so the pairs at work share a few weight tiles and x stays in L2.
// Up to 192 tokens a tile, TMEM holds two tiles' accumulators and the epilogue
// of one runs beside the MMAs of the next; with 256 tokens it holds one.
// Roles of a CTA's fourteen warps:
//   0-7   epilogue: 32 tokens x 32 outputs at a time from TMEM to the warp's
//         shared memory in the output's type, and from there to y by TMA
//         (straight to y where its rows are not 16-byte aligned);
//   8-11  scales to TMEM;
//   12    one thread: the codes by TMA, into this CTA's ring; both CTAs' copies
//         complete on the first CTA's `full` barriers, where the scale warps
//         of both arrive too;
//   13    one thread of the first CTA: MMAs for the pair; tcgen05.commit
//         returns a stage, or hands over a tile, in both CTAs.
// Measured (B200, graph replay, the tokens' quantising included): 4096 tokens of
// 5120 x 27648, bf16 out, 289 us (4.0 PFLOP/s); 1111 of 4096 x 12288, 43.9 us (2.5
// PFLOP/s: four rounds of tiles, the last nine tenths full, and about 9 us of
// quantising, the scales' pass, ramp and last epilogue).  Bound by the copies out of L2: 36 bytes a clock reach an SM when
// all ask, 800 clocks for a stage whose MMAs take 440 (NT = 192).
//
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

constexpr int kPThreads = 448;
constexpr int kChunk = 32;     // tokens an epilogue warp takes at a time
constexpr int kOutRing = 2;    // its chunks on their way to y
constexpr int kSfAhead = 2;    // stages whose scales are in flight
using mx4::kStageK;

template <int NT>
struct PCfg {
  static constexpr int kHalves = (NT + 127) / 128;  // 128-token runs of scales
  static constexpr int kAcc = NT <= 192 ? 2 : 1;    // tiles whose accumulators TMEM holds
  static constexpr int kStages = NT == 128 ? 6 : 5;
  static constexpr uint32_t kA = 128 * 128, kB = NT / 2 * 128;
  static constexpr uint32_t kStage = kA + kB;
  static constexpr uint32_t kOut = kChunk * 32 * 4;  // a chunk of outputs (fp32)
  static constexpr int kSfCols = 8 + 8 * kHalves;     // TMEM columns of a stage's scales
  static constexpr int kTmemCols = 512;
  static constexpr size_t kSmem = (size_t)kStages * kStage + 8 * kOutRing * kOut + 1024;
  static_assert(kStage % 1024 == 0, "swizzled stages stay 1024-byte aligned");
  static_assert(kAcc * NT + kStages * kSfCols <= kTmemCols, "TMEM");
  static_assert(kSmem <= 227 * 1024, "shared memory");
};

struct PParams {
  void* y;
  int out_bf16;
  const uint4* ws;  // arranged scales of the weight, then of x
  const uint4* xs;
  int M, d_in, d_out;
  int tn, tiles;  // token tiles, all tiles
  int tma_out;    // y's rows are 16-byte aligned: map_y stores them
  int* dev_status;
  unsigned long long wait_ns;
};

// Address of this CTA's shared variable in the first CTA of the pair.
__device__ __forceinline__ uint32_t in_first(const void* p) {
  uint32_t a;
  asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(a) : "r"(smem_u32(p)));
  return a;
}

// Arrives at a barrier of the pair.  What it announces lies in TMEM and is
// ordered by the tcgen05 fences around it, so the arrival itself orders
// nothing: with release semantics at cluster scope it took about 1700 clocks.
__device__ __forceinline__ void arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// A whole warp waits for a phase: one lane asks, so that the others' questions
// do not take the shared memory's time.  The same answer in every lane.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort,
                                          unsigned long long limit_ns) {
  bool ok = true;
  if ((threadIdx.x & 31) == 0) ok = mx4::wait_bounded<16>(bar, parity, abort, limit_ns);
  return __shfl_sync(0xffffffffu, (int)ok, 0) != 0;
}

// TMA tile to this CTA's shared memory, completing on a barrier of the pair.
__device__ __forceinline__ void tma_load_pair(void* dst, const CUtensorMap* map, int c0, int c1, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
      " [%0], [%1, {%3, %4}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1)
      : "memory");
}

// Eight or sixteen words of every lane to consecutive TMEM columns.
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t* w) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr),
               "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* w) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16};" ::"r"(taddr),
      "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7]), "r"(w[8]), "r"(w[9]),
      "r"(w[10]), "r"(w[11]), "r"(w[12]), "r"(w[13]), "r"(w[14]), "r"(w[15])
      : "memory");
}

// A tile of shared memory to global memory by TMA (one thread).
__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, int c0, int c1, const void* src) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(smem_u32(src)), "r"(c0), "r"(c1)
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

template <int NT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPThreads, 1)
    mx4_pair_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x,
                    const __grid_constant__ CUtensorMap map_y, const PParams p) {
  using C = PCfg<NT>;
  constexpr int kS = C::kStages;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* stages = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ uint64_t full[kS], empty[kS], acc_full[C::kAcc], acc_empty[C::kAcc];
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;

  cg::cluster_group cluster = cg::this_cluster();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = static_cast<int>(cluster.block_rank());
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  const int n_it = (p.d_in + kStageK - 1) / kStageK;

  if (tid == 0) {
    for (int s = 0; s < kS; ++s) {
      mbar_init(&full[s], 1 + 8);  // the first CTA's TMA thread (and both CTAs' bytes), both CTAs' scale warps
      mbar_init(&empty[s], 1);
    }
    for (int i = 0; i < C::kAcc; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], 16);  // both CTAs' epilogue warps
    }
    s_abort = 0;
    mbar_init_fence();
  }
  if (warp == 13) {
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

  if (warp < 8) {
    // ---------------------------------------------------------------- epilogue
    // warp w: TMEM lanes 32 (w % 4) ..., half w / 4 of the tokens
    const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    unsigned char* ring = stages + (size_t)kS * C::kStage + (size_t)warp * kOutRing * C::kOut;
    int round = 0, chunk_no = 0;
    for (int tile = pair; tile < p.tiles; tile += pairs, ++round) {
      const int n0 = tile % p.tn * NT, j0 = tile / p.tn * 256 + rank * 128 + (warp & 3) * 32;
      const int acc = round % C::kAcc;
      if (!warp_wait(&acc_full[acc], (uint32_t)(round / C::kAcc) & 1u, abort_flag, p.wait_ns)) {
        *abort_flag = 1;
        break;
      }
      tc::tmem_fence_after();
      const int begin = warp < 4 ? 0 : NT / 2, end = begin + NT / 2;
#pragma unroll 1
      for (int c0 = begin; c0 < end; c0 += kChunk, ++chunk_no) {
        float v[kChunk];
        tc::tmem_ld32(lanes + acc * NT + c0, v);
        if (c0 + kChunk >= end) {  // this warp's accumulators are read: their next tile may start
          tc::tmem_fence_before();
          __syncwarp();
          if (lane == 0) arrive_cluster(in_first(&acc_empty[acc]));
        }
        if (p.tma_out) {
          // [token][32 outputs]; the chunk that was here before has left
          unsigned char* out = ring + (size_t)(chunk_no % kOutRing) * C::kOut;
          if (lane == 0) asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(kOutRing - 1) : "memory");
          __syncwarp();
          if (p.out_bf16) {
            __nv_bfloat16* at = reinterpret_cast<__nv_bfloat16*>(out) + lane;
#pragma unroll
            for (int c = 0; c < kChunk; ++c) at[c * 32] = __float2bfloat16_rn(v[c]);  // the caller's output type
          } else {
            float* at = reinterpret_cast<float*>(out) + lane;
#pragma unroll
            for (int c = 0; c < kChunk; ++c) at[c * 32] = v[c];
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          if (lane == 0) {  // what lies past y is not written; a group per chunk all the same
            if (j0 < p.d_out && n0 + c0 < p.M) tma_store_2d(&map_y, j0, n0 + c0, out);
            asm volatile("cp.async.bulk.commit_group;" ::: "memory");
          }
        } else if (j0 + lane < p.d_out) {
          const size_t at = (size_t)(n0 + c0) * p.d_out + j0 + lane;
          const int tokens = min(kChunk, p.M - n0 - c0);
#pragma unroll
          for (int c = 0; c < kChunk; ++c)
            if (c < tokens) {
              if (p.out_bf16)
                static_cast<__nv_bfloat16*>(p.y)[at + (size_t)c * p.d_out] = __float2bfloat16_rn(v[c]);
              else
                static_cast<float*>(p.y)[at + (size_t)c * p.d_out] = v[c];
            }
        }
      }
    }
    // every store has read its shared memory before the CTA leaves
    if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  } else if (warp < 12) {
    // ---------------------------------------------------------------- scales
    const int mine = p.tiles > pair ? (p.tiles - pair + pairs - 1) / pairs : 0;
    const int total = mine * n_it;
    const uint32_t cols = tmem + ((uint32_t)((warp & 3) * 32) << 16) + C::kAcc * NT;
    constexpr int kWords = 2 + 2 * C::kHalves;  // 16-byte words of a lane and stage
    uint4 w[kSfAhead][kWords];
    int l_tile = pair, l_it = 0;  // the next stage to load
    auto load = [&](int u) {
      if (l_tile >= p.tiles) return;
      const uint4* a = p.ws + ((size_t)(l_tile / p.tn * 2 + rank) * n_it + l_it) * 64 + lane;
      const uint4* b = p.xs + ((size_t)(l_tile % p.tn) * n_it + l_it) * (64 * C::kHalves) + lane;
      w[u][0] = __ldg(a);
      w[u][1] = __ldg(a + 32);
#pragma unroll
      for (int i = 0; i < 2 * C::kHalves; ++i) w[u][2 + i] = __ldg(b + 32 * i);
      if (++l_it == n_it) {
        l_it = 0;
        l_tile += pairs;
      }
    };
#pragma unroll
    for (int u = 0; u < kSfAhead; ++u) load(u);
    bool ok = true;  // the same in every lane
    int s = 0, use = 0;
    for (int base = 0; base < total && ok; base += kSfAhead) {
#pragma unroll
      for (int u = 0; u < kSfAhead; ++u) {
        if (base + u >= total || !ok) break;
        if (use > 0) {
          ok = warp_wait(&empty[s], (uint32_t)(use - 1) & 1u, abort_flag, p.wait_ns);
          if (!ok) {
            *abort_flag = 1;
            break;
          }
        }
        tc::tmem_fence_after();
        uint32_t words[4 * kWords];
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
          words[4 * i] = w[u][i].x;
          words[4 * i + 1] = w[u][i].y;
          words[4 * i + 2] = w[u][i].z;
          words[4 * i + 3] = w[u][i].w;
        }
        tmem_st16(cols + s * C::kSfCols, words);
        if constexpr (C::kHalves == 2) tmem_st8(cols + s * C::kSfCols + 16, words + 16);
        load(u);
        asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
        tc::tmem_fence_before();
        __syncwarp();
        if (lane == 0) arrive_cluster(in_first(&full[s]));
        if (++s == kS) {
          s = 0;
          ++use;
        }
      }
    }
  } else if (warp == 12) {
    // ---------------------------------------------------------------- codes
    if (lane == 0) {
      int s = 0, use = 0;
      bool ok = true;
      for (int tile = pair; tile < p.tiles && ok; tile += pairs) {
        const int n0 = tile % p.tn * NT, j0 = tile / p.tn * 256;
        for (int it = 0; it < n_it; ++it) {
          if (use > 0 && !mx4::wait_bounded<16>(&empty[s], (uint32_t)(use - 1) & 1u, abort_flag, p.wait_ns)) {
            *abort_flag = 1;
            ok = false;
            break;
          }
          unsigned char* dst = stages + (size_t)s * C::kStage;
          if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * C::kStage);  // both CTAs' copies
          const uint32_t bar = in_first(&full[s]);
          tma_load_pair(dst, &map_w, it * 128, j0 + rank * 128, bar);
          tma_load_pair(dst + C::kA, &map_x, it * 128, n0 + rank * (NT / 2), bar);
          if (++s == kS) {
            s = 0;
            ++use;
          }
        }
      }
    }
  } else if (rank == 0) {
    // ---------------------------------------------------------------- MMA issuer
    if (lane == 0) {
      int s = 0, use = 0, round = 0;
      bool ok = true;
      for (int tile = pair; tile < p.tiles && ok; tile += pairs, ++round) {
        const int acc = round % C::kAcc;
        if (round >= C::kAcc &&
            !mx4::wait_bounded<16>(&acc_empty[acc], (uint32_t)(round / C::kAcc - 1) & 1u, abort_flag, p.wait_ns)) {
          *abort_flag = 1;
          break;
        }
        tc::tmem_fence_after();
        for (int it = 0; it < n_it; ++it) {
          if (!mx4::wait_bounded<16>(&full[s], (uint32_t)use & 1u, abort_flag, p.wait_ns)) {
            *abort_flag = 1;
            ok = false;
            break;
          }
          tc::tmem_fence_after();
          const uint32_t a_addr = smem_u32(stages + (size_t)s * C::kStage), b_addr = a_addr + C::kA;
          // this stage's scale columns: weight 4 + 4, then tokens
          const uint32_t ta = tmem + C::kAcc * NT + s * C::kSfCols, tb = ta + 8;
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)  // 64 inputs (32 bytes) each
            mx4::umma_mxf4<2>(tmem + acc * NT, tc::sw128_desc(a_addr + kk * 32), tc::sw128_desc(b_addr + kk * 32),
                              mx4::idesc_mxf4(256, NT, 2 * (kk & 1)), ta + 4 * (kk >> 1),
                              tb + 4 * C::kHalves * (kk >> 1), (it > 0 || kk > 0) ? 1u : 0u);
          commit_pair(&empty[s]);
          if (++s == kS) {
            s = 0;
            ++use;
          }
        }
        if (ok) commit_pair(&acc_full[acc]);
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
  if (*abort_flag || *cluster.map_shared_rank(&s_abort, 1 - rank)) {
    // what was issued for the pair ends before its memory goes away; a stage
    // that was given up has no barrier that would tell
    const unsigned long long t0 = global_timer_ns();
    while (global_timer_ns() - t0 < mx4::kSettleNs) {
    }
    __syncthreads();
  }
  if (warp == 13) {
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

// A tensor map of y, boxes of 32 tokens x 32 outputs.
bool make_out_map(CUtensorMap* map, void* y, bool bf16, int M, int d_out) {
  const tc::EncodeTiled enc = tc::encoder();
  if (enc == nullptr) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)d_out, (cuuint64_t)M};
  const cuuint64_t strides[1] = {(cuuint64_t)d_out * (bf16 ? 2 : 4)};
  const cuuint32_t box[2] = {32, kChunk};
  const cuuint32_t estr[2] = {1, 1};
  return enc(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, y, dims, strides, box,
             estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_NONE,
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
  const long long w_rows = weight_runs(p.d_out) * n_it;
  unsigned char* wbuf = static_cast<unsigned char*>(buf);
  unsigned char* xbuf = wbuf + w_rows * 1024;
  p.ws = reinterpret_cast<const uint4*>(wbuf);
  p.xs = reinterpret_cast<const uint4*>(xbuf);
  p.tma_out = ((size_t)p.d_out * (p.out_bf16 ? 2 : 4)) % 16 == 0;
  CUtensorMap map_w, map_x, map_y = {};
  if (!mx4::make_byte_map(&map_w, wc, p.d_out, p.d_in / 2, 128) ||
      !mx4::make_byte_map(&map_x, xc, p.M, p.d_in / 2, NT / 2) ||
      (p.tma_out && !make_out_map(&map_y, p.y, p.out_bf16 != 0, p.M, p.d_out)))
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
  return cudaLaunchKernelEx(&cfg, mx4_pair_kernel<NT>, map_w, map_x, map_y, p);
}

}  // namespace

// Clocks of a shape with NT tokens per tile: rounds of the pairs times a
// tile's stages (its MMAs, or its copies at the 36 bytes per clock and SM that
// L2 gives when every SM asks, whichever takes longer), and the epilogue where
// nothing hides it.
double mx4_pair_clocks(int nt, int M, int d_in, int d_out) {
  const long long tiles = (long long)((M + nt - 1) / nt) * ((d_out + 255) / 256);
  const int n_it = (d_in + kStageK - 1) / kStageK;
  const double epilogue = 300.0 * nt / (2 * kChunk);
  const double main = n_it * std::max(2.0 * nt + 60.0, (16384.0 + 64.0 * nt) / 36.0);
  const double tile = nt <= 192 ? std::max(main, epilogue) : main + epilogue;
  return (double)((tiles + 73) / 74) * tile + epilogue + 9000.0;  // 9000: the scales' pass and a ramp
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
  PParams p{y, out_bf16 ? 1 : 0, nullptr, nullptr, M, d_in, d_out, 0, 0, 0, dev_status, wait_limit_ns()};
  switch (nt) {
    case 128: return launch_pair_nt<128>(x_codes, x_scales, w_codes, w_scales, buf, p, stream);
    case 192: return launch_pair_nt<192>(x_codes, x_scales, w_codes, w_scales, buf, p, stream);
    default: return launch_pair_nt<256>(x_codes, x_scales, w_codes, w_scales, buf, p, stream);
  }
}

}  // namespace larosa
