// Building blocks of the kernels that multiply MX4 matrices on the
// fifth-generation tensor cores (tcgen05 kind::mxf4 with block scales).
#pragma once

#include "mx4.cuh"
#include "tcgen05.cuh"

namespace larosa {
namespace mx4 {

constexpr int kStageK = 256;  // inputs per pipeline stage: 128-byte rows of codes, the swizzle width
constexpr int kStageBlocks = kStageK / kBlock;

// How long a kernel that gives up lets the copies and MMAs it has issued end
// before it frees what they use, whatever the wait limit: they take
// microseconds, and the limit may be as short as one.
constexpr unsigned long long kSettleNs = 100000;

// mbar_wait_bounded that looks at the clock and at *abort every kEvery tries: the
// hardware holds a try for a fraction of a microsecond, so that the 256 tries
// between two looks there outlast the shortest limits (at 1 us no wait of a
// product of 3 tokens of 32768 x 20000 ran out; so every call's does).  One try for
// the stages of few tokens, 12.0 us for 3 of 11008 x 4096 (12.1 with 256); 16 for the
// pairs of SMs, 290.5 us for 4096 of 5120 x 27648 as with 256 (291.4 with one).
template <uint32_t kEvery>
__device__ __forceinline__ bool wait_bounded(uint64_t* bar, uint32_t parity, volatile int* abort,
                                             unsigned long long limit_ns) {
  if (mbar_try_wait(bar, parity)) return true;
  const unsigned long long t0 = global_timer_ns();
  for (uint32_t it = 1; !mbar_try_wait(bar, parity); ++it)
    if (it % kEvery == 0 && ((abort != nullptr && *abort) || global_timer_ns() - t0 > limit_ns)) return false;
  return true;
}

// Instruction descriptor of kind::mxf4: A and B e2m1 (1), K-major, scales
// ue8m0, M = m, N = n; sf selects which half of a scale word the 64 inputs
// take (0: bytes 0-1, 2: bytes 2-3).
constexpr uint32_t idesc_mxf4(int m, int n, int sf) {
  return ((uint32_t)sf << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) | (1u << 23) |
         ((uint32_t)(m >> 7) << 27) | ((uint32_t)sf << 29);
}

// D += A B over 64 inputs, kGroup CTAs (two: M = 256, 128 rows of A and half
// of B's columns in each).
template <int kGroup>
__device__ __forceinline__ void umma_mxf4(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t sfa, uint32_t sfb,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::%7.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(id), "r"(sfa), "r"(sfb), "r"(accumulate), "n"(kGroup)
      : "memory");
}

// 512 bytes of scales (32 rows of 16 bytes) to four TMEM columns, in every
// warp's lanes.  Descriptor: no swizzle, groups of eight rows 128 bytes apart.
__device__ __forceinline__ void copy_scales(uint32_t tmem, uint32_t saddr) {
  const uint64_t desc = (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)1 << 16) | ((uint64_t)(128 >> 4) << 32) |
                        ((uint64_t)1 << 46);
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(desc) : "memory");
}

// Eight scale bytes of a row from block kb on; zeros past the row's end.
__device__ __forceinline__ uint2 load_scales(const uint8_t* row, int blocks, int kb) {
  if (row == nullptr || kb >= blocks) return make_uint2(0u, 0u);
  if ((blocks & 7) == 0) return __ldg(reinterpret_cast<const uint2*>(row + kb));  // rows 8-byte aligned
  uint32_t w[2] = {0u, 0u};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (kb + i < blocks) w[i >> 2] |= (uint32_t)__ldg(row + kb + i) << (8 * (i & 3));
  return make_uint2(w[0], w[1]);
}

// A 2-D byte tensor map of a row-major [rows x bytes] matrix, box
// [box_rows x 128 bytes], 128-byte swizzle.
inline bool make_byte_map(CUtensorMap* map, const void* base, int rows, int bytes, int box_rows) {
  const tc::EncodeTiled enc = tc::encoder();
  if (enc == nullptr) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)bytes, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)bytes};
  const cuuint32_t box[2] = {128u, (cuuint32_t)box_rows};
  const cuuint32_t estr[2] = {1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace mx4
}  // namespace larosa
