// Product of two microscaled 4-bit matrices (sm_100a), one token to a prompt:
//
//   y[m][j] = sum_i x[m][i] W[j][i],  x [M x d_in], W [d_out x d_in]
//   (torch.nn.Linear layout), both MX4 with blocks along d_in (mx4.cuh):
//   every 32 products of 4-bit values are scaled by 2^(bx + bw - 254).
//
// The fifth-generation tensor cores multiply this format as it is
// (tcgen05.mma kind::mxf4 with block scales, 64 inputs per instruction, four
// times the bf16 rate): nothing is decoded.  The weight's rows are the M = 128
// side of an MMA tile, the tokens its N side, so that a warp of the epilogue
// holds 32 neighbouring outputs of a token and stores them together; fp32
// accumulators in TMEM.
//
// A CTA owns 128 outputs x NT tokens and one split of the reduction, in
// stages of 256 inputs (128-byte rows of codes, the swizzle width):
//   * one thread brings the codes of both tiles in by TMA (2-D tile copies,
//     128-byte swizzle; what lies past the matrix arrives as zeros);
//   * four warps bring the scale bytes: thread r the eight of weight row r
//     and of token r, loaded four stages ahead and stored in the order the
//     tensor core reads scales in (512 bytes for 128 rows x 4 blocks: row r at
//     16 (r % 32) + 4 (r / 32)).  The row-major scales of the format are read
//     as they are, eight bytes of a row at a time;
//   * one thread copies a stage's scales into TMEM (tcgen05.cp) and issues its
//     four MMAs; tcgen05.commit returns the stage;
//   * the four warps then read the accumulators.
// The splits of a tile (few tokens: the weight's bytes must come through every
// SM) form a thread-block cluster and add their partial tiles through
// distributed shared memory in rank order, so results do not depend on
// timing.  Every wait is bounded, as in the other tensor-core kernels.
//
// This kernel takes up to 64 tokens per tile; from there on pairs of SMs
// share a tile (mx4_pair.cu).  Tokens vary fastest over the grid, so the CTAs
// at work share weight tiles.
//
// Measured (B200, graph replay, from HBM, the tokens' quantising included): 3
// tokens of 11008 x 4096, 12.1 us (24 MB, 2.0 TB/s): more than half is the way in
// and out, the launches, TMEM, the first stage's latency and the splits' sum.
#include <cooperative_groups.h>
#include <cuda.h>

#include <algorithm>

#include "common.cuh"
#include "internal.h"
#include "mx4.cuh"
#include "mx4_umma.cuh"

namespace cg = cooperative_groups;

namespace larosa {
namespace {

constexpr int kLThreads = 192;  // warps 0-3: scales, then epilogue; 4: TMA; 5: MMA
constexpr int kRows = 128;      // outputs per CTA
constexpr int kAhead = 4;       // stages whose scales are in flight
using mx4::kStageBlocks;
using mx4::kStageK;

template <int NT>
struct LCfg {
  static constexpr int kStages = NT == 16 ? 5 : 4;
  static constexpr int kPerSm = 2;  // CTAs an SM holds
  static constexpr uint32_t kA = kRows * 128, kB = NT * 128;
  static constexpr uint32_t kSfA = 1024, kSfB = 1024;
  static constexpr uint32_t kStage = kA + kB + kSfA + kSfB;
  static constexpr int kSfCols = 8 + 8;  // TMEM columns of a stage's scales
  static constexpr int kD = NT < 32 ? 32 : NT;
  static constexpr int kTmemUsed = kD + kStages * kSfCols;
  static constexpr int kTmemCols = kTmemUsed <= 128 ? 128 : kTmemUsed <= 256 ? 256 : 512;
  static constexpr size_t kSmem = (size_t)kStages * kStage + 1024;
  static_assert(kStage % 1024 == 0, "swizzled stages stay 1024-byte aligned");
  static_assert(kTmemUsed <= 512 && kPerSm * kTmemCols <= 512, "TMEM");
  static_assert((size_t)NT * kRows * 4 <= (size_t)kStages * kStage, "partials fit the ring");
};

struct LParams {
  const uint8_t* xs;  // scales of x [M x d_in / 32]
  const uint8_t* ws;  // scales of W [d_out x d_in / 32]
  void* y;
  int out_bf16;
  int M, d_in, d_out;
  int stages_per_split;
  int* dev_status;
  unsigned long long wait_ns;
};

__device__ __forceinline__ void store_out(const LParams& p, size_t at, float v) {
  if (p.out_bf16)
    static_cast<__nv_bfloat16*>(p.y)[at] = __float2bfloat16_rn(v);  // the caller's output type
  else
    static_cast<float*>(p.y)[at] = v;
}

template <int NT>
__global__ void __launch_bounds__(kLThreads, 1)
    mx4_linear_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x,
                      const LParams p) {
  using C = LCfg<NT>;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* stages = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ uint64_t full[C::kStages], empty[C::kStages], done;
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int split = blockIdx.x;  // = rank in the cluster
  const int n0 = blockIdx.y * NT, j0 = blockIdx.z * kRows;
  const int total = (p.d_in + kStageK - 1) / kStageK;
  const int it0 = split * p.stages_per_split;
  const int n_it = max(0, min(total, it0 + p.stages_per_split) - it0);

  if (tid == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&full[s], 1 + 4);  // the TMA thread and the four scale warps
      mbar_init(&empty[s], 1);
    }
    mbar_init(&done, 1);
    s_abort = 0;
    mbar_init_fence();
  }
  if (warp == 5) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s_tmem)),
                 "r"(C::kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc::tmem_fence_before();
  __syncthreads();
  tc::tmem_fence_after();
  const uint32_t tmem = s_tmem;
  volatile int* abort_flag = &s_abort;

  // codes and scales may have been written by the kernel before this one
  // (larosa_mx4_quantize lets this one start early)
  pdl_wait();
  pdl_launch_dependents();

  int issued = 0;  // stages whose copies this thread (warp 4, lane 0) has armed
  if (warp < 4) {
    // ---------------------------------------------------------------- scales
    const int blocks = p.d_in / mx4::kBlock;
    const uint8_t* wrow = j0 + tid < p.d_out ? p.ws + (size_t)(j0 + tid) * blocks : nullptr;
    const uint8_t* xrow = tid < NT && n0 + tid < p.M ? p.xs + (size_t)(n0 + tid) * blocks : nullptr;
    uint2 a[kAhead], b[kAhead];
    auto load = [&](int it, int u) {
      const int kb = it < n_it ? (it0 + it) * kStageBlocks : blocks;
      a[u] = mx4::load_scales(wrow, blocks, kb);
      b[u] = mx4::load_scales(xrow, blocks, kb);
    };
#pragma unroll
    for (int u = 0; u < kAhead; ++u) load(u, u);
    const uint32_t at = 16 * (tid & 31) + 4 * (tid >> 5);
    bool ok = true;  // the same in every lane
    for (int base = 0; base < n_it && ok; base += kAhead) {
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int it = base + u;
        if (it >= n_it || !ok) break;
        const int s = it % C::kStages;
        if (it >= C::kStages) {
          ok = mx4::wait_bounded<1>(&empty[s], ((it / C::kStages) - 1) & 1, abort_flag, p.wait_ns);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) {
            *abort_flag = 1;
            break;
          }
        }
        unsigned char* sfa = stages + (size_t)s * C::kStage + C::kA + C::kB;
        unsigned char* sfb = sfa + C::kSfA;
        *reinterpret_cast<uint32_t*>(sfa + at) = a[u].x;
        *reinterpret_cast<uint32_t*>(sfa + 512 + at) = a[u].y;
        *reinterpret_cast<uint32_t*>(sfb + at) = b[u].x;
        *reinterpret_cast<uint32_t*>(sfb + 512 + at) = b[u].y;
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) mbar_arrive(&full[s]);
        load(it + kAhead, u);
      }
    }
  } else if (warp == 4) {
    // ---------------------------------------------------------------- codes
    if (lane == 0) {
      for (int it = 0; it < n_it; ++it) {
        const int s = it % C::kStages;
        if (it >= C::kStages && !mx4::wait_bounded<1>(&empty[s], ((it / C::kStages) - 1) & 1, abort_flag, p.wait_ns)) {
          *abort_flag = 1;
          break;
        }
        unsigned char* dst = stages + (size_t)s * C::kStage;
        mbar_arrive_expect_tx(&full[s], C::kA + C::kB);
        tc::tma_load_2d(dst, &map_w, (it0 + it) * 128, j0, &full[s]);
        tc::tma_load_2d(dst + C::kA, &map_x, (it0 + it) * 128, n0, &full[s]);
        ++issued;
      }
    }
  } else {
    // ---------------------------------------------------------------- MMA issuer
    if (lane == 0) {
      for (int it = 0; it < n_it; ++it) {
        const int s = it % C::kStages;
        if (!mx4::wait_bounded<1>(&full[s], (it / C::kStages) & 1, abort_flag, p.wait_ns)) {
          *abort_flag = 1;
          break;
        }
        tc::tmem_fence_after();
        const uint32_t a_addr = smem_u32(stages + (size_t)s * C::kStage);
        const uint32_t b_addr = a_addr + C::kA, sfa = b_addr + C::kB, sfb = sfa + C::kSfA;
        // this stage's scale columns: weight 4 + 4, then tokens
        const uint32_t ta = tmem + C::kD + s * C::kSfCols, tb = ta + 8;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          mx4::copy_scales(ta + 4 * c, sfa + 512 * c);
          mx4::copy_scales(tb + 4 * c, sfb + 512 * c);
        }
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)  // 64 inputs (32 bytes) each
          mx4::umma_mxf4<1>(tmem, tc::sw128_desc(a_addr + kk * 32), tc::sw128_desc(b_addr + kk * 32),
                    mx4::idesc_mxf4(128, NT, 2 * (kk & 1)), ta + 4 * (kk >> 1), tb + 4 * (kk >> 1),
                    (it > 0 || kk > 0) ? 1u : 0u);
        tc::umma_commit(&empty[s]);  // the stage is free once these MMAs have read it
      }
      tc::umma_commit(&done);  // every MMA issued above has completed
    }
  }
  __syncwarp();

  // ------------------------------------------------------------------ epilogue
  const bool finished = mx4::wait_bounded<1>(&done, 0, nullptr, p.wait_ns);
  tc::tmem_fence_after();
  __syncwarp();  // tcgen05.ld is .aligned: the whole warp issues it together
  if (!finished) *abort_flag = 1;
  __syncthreads();
  if (*abort_flag && warp == 4 && lane == 0) {
    // let the MMAs and every copy this CTA armed end before its memory goes
    // away; a stage whose scales never came cannot complete and takes the whole
    // time
    mx4::wait_bounded<1>(&done, 0, nullptr, mx4::kSettleNs);
    for (int it = max(0, issued - C::kStages); it < issued; ++it)
      mx4::wait_bounded<1>(&full[it % C::kStages], (it / C::kStages) & 1, nullptr, mx4::kSettleNs);
    report(p.dev_status, LAROSA_DEV_TIMEOUT);
  }
  __syncthreads();
  const bool abort = *abort_flag != 0;
  constexpr int kChunk = NT < 32 ? 16 : 32;  // accumulator columns at a time
  const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
  const int R = static_cast<int>(gridDim.x);
  if (R == 1) {
    if (warp < 4 && !abort) {
      const int j = j0 + tid;
#pragma unroll 1
      for (int c0 = 0; c0 < NT && n0 + c0 < p.M; c0 += kChunk) {
        float v[kChunk];
        if constexpr (kChunk == 16)
          tc::tmem_ld16(lanes + c0, v);
        else
          tc::tmem_ld32(lanes + c0, v);
        if (j < p.d_out) {
          const size_t at = (size_t)(n0 + c0) * p.d_out + j;
          const int n = min(kChunk, p.M - n0 - c0);
#pragma unroll
          for (int c = 0; c < kChunk; ++c)
            if (c < n) store_out(p, at + (size_t)c * p.d_out, v[c]);
        }
      }
    }
    tc::tmem_fence_before();
    __syncthreads();
    if (warp == 5) {
      tc::tmem_fence_after();
      asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(C::kTmemCols) : "memory");
    }
    return;
  }
  // the splits' partial tiles, [token][output] in the (now idle) ring
  {
    cg::cluster_group cluster = cg::this_cluster();
    float* part = reinterpret_cast<float*>(stages);
    if (warp < 4) {
#pragma unroll 1
      for (int c0 = 0; c0 < NT; c0 += kChunk) {
        float v[kChunk];
        if constexpr (kChunk == 16)
          tc::tmem_ld16(lanes + c0, v);
        else
          tc::tmem_ld32(lanes + c0, v);
#pragma unroll
        for (int c = 0; c < kChunk; ++c) part[(c0 + c) * kRows + tid] = n_it > 0 ? v[c] : 0.f;
      }
    }
    tc::tmem_fence_before();
    __syncthreads();
    if (warp == 5) {
      tc::tmem_fence_after();
      asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(C::kTmemCols) : "memory");
    }
    cluster.sync();
    if (!abort) {
      const int r0 = split * kRows / R, rows = (split + 1) * kRows / R - r0;
      const int n = rows * min(NT, p.M - n0);
      for (int e = tid; e < n; e += kLThreads) {
        const int m = e / rows, row = r0 + e % rows;
        float s = 0.f;
        for (int q = 0; q < R; ++q) s += cluster.map_shared_rank(part, q)[m * kRows + row];
        if (j0 + row < p.d_out) store_out(p, (size_t)(n0 + m) * p.d_out + j0 + row, s);
      }
    }
    cluster.sync();  // no CTA leaves while another may still read its partial tile
  }
}

template <int NT>
cudaError_t launch_nt(const void* xc, const void* wc, LParams p, int R, cudaStream_t stream) {
  using C = LCfg<NT>;
  static int configured[64] = {0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!configured[dev]) {
    e = cudaFuncSetAttribute(mx4_linear_kernel<NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::kSmem);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(mx4_linear_kernel<NT>, cudaFuncAttributePreferredSharedMemoryCarveout,
                               cudaSharedmemCarveoutMaxShared);
    if (e != cudaSuccess) return e;
    configured[dev] = 1;
  }
  CUtensorMap map_w, map_x;
  if (!mx4::make_byte_map(&map_w, wc, p.d_out, p.d_in / 2, kRows) || !mx4::make_byte_map(&map_x, xc, p.M, p.d_in / 2, NT))
    return cudaErrorInvalidValue;
  const int total = (p.d_in + kStageK - 1) / kStageK;
  p.stages_per_split = (total + R - 1) / R;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(R, (p.M + NT - 1) / NT, (p.d_out + kRows - 1) / kRows);
  cfg.blockDim = dim3(kLThreads, 1, 1);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = R;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, mx4_linear_kernel<NT>, map_w, map_x, p);
}

// Clocks of a shape with NT tokens per tile and R splits: full waves of CTAs
// times a CTA's stages, each as long as its copies at 42 bytes per clock and
// SM or its MMAs, and a fixed part.
template <int NT>
double tile_clocks(int M, int d_in, int d_out, int R) {
  using C = LCfg<NT>;
  const int total = (d_in + kStageK - 1) / kStageK;
  const long long ctas = (long long)((M + NT - 1) / NT) * ((d_out + kRows - 1) / kRows) * R;
  const long long slots = 148LL * C::kPerSm;
  const long long waves = (ctas + slots - 1) / slots;
  const double stage = std::max(2.0 * NT, C::kStage / 42.0) * C::kPerSm;
  return (double)waves * (((total + R - 1) / R) * stage + 4000.0 + 20.0 * NT);
}

}  // namespace

// Tokens from which pairs of SMs are considered.
constexpr int kPairTokens = 65;

size_t mx4_linear_buffer_bytes(int M, int d_in, int d_out) {
  return M < kPairTokens ? 0 : mx4_pair_buffer_bytes(M, d_in, d_out);
}

cudaError_t launch_mx4_linear(const void* x_codes, const void* x_scales, const void* w_codes, const void* w_scales,
                              int M, int d_in, int d_out, void* y, bool out_bf16, void* buf, int* dev_status,
                              cudaStream_t stream) {
  LParams p{static_cast<const uint8_t*>(x_scales), static_cast<const uint8_t*>(w_scales), y, out_bf16 ? 1 : 0,
            M, d_in, d_out, 0, dev_status, wait_limit_ns()};
  const int total = (d_in + kStageK - 1) / kStageK;
  // The tile and split that the model puts first; splits only of tiles of up
  // to 64 tokens, at most 8 (the portable cluster size).  Tiles of 128 tokens
  // and more run on pairs of SMs (mx4_pair.cu).
  int nt = 0, R = 1;
  double best = 0.0;
  auto consider = [&](int n, int r, double t) {
    if (nt == 0 || t < best) {
      nt = n;
      R = r;
      best = t;
    }
  };
  for (int r = 1; r <= 8 && r <= total; r *= 2) {
    if (M <= 16) consider(16, r, tile_clocks<16>(M, d_in, d_out, r));
    consider(32, r, tile_clocks<32>(M, d_in, d_out, r));
    if (M > 32) consider(64, r, tile_clocks<64>(M, d_in, d_out, r));
  }
  for (int n : {128, 192, 256})
    if (M >= kPairTokens) consider(n, 1, mx4_pair_clocks(n, M, d_in, d_out));
  switch (nt) {
    case 16: return launch_nt<16>(x_codes, w_codes, p, R, stream);
    case 32: return launch_nt<32>(x_codes, w_codes, p, R, stream);
    case 64: return launch_nt<64>(x_codes, w_codes, p, R, stream);
    default:
      return launch_mx4_pair(nt, x_codes, x_scales, w_codes, w_scales, M, d_in, d_out, y, out_bf16, buf, dev_status,
                             stream);
  }
}

}  // namespace larosa
