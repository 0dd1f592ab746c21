// Products of a few tokens with rows of a 4-bit (MX4) weight on mma.sync,
// shared by the sparse linear and the expert layer: see mx4_rows.cu for the
// arithmetic.  A warp multiplies blocks of 32 rows by 128 columns; lane
// (g, t) = (lane / 4, lane % 4) holds the columns 16 g .. 16 g + 15 of the
// rows 4 t .. 4 t + 3 of a 16-row step.
#pragma once

#include "mx4.cuh"

namespace larosa {
namespace mx4 {

// Powers of two that take a block of fp32 values with largest magnitude bits
// `top` into [2^14, 2^15) and back: v * up, (...) * down.  The exponent is
// held at -100 or above, so that both are normal numbers; a smaller block
// keeps its absolute error.
__device__ __forceinline__ void piece_scale(unsigned top, float* up, float* down) {
  const int e = max(static_cast<int>(top >> 23) - 127, -100);  // 128 for a NaN or Inf block
  *up = __uint_as_float(static_cast<unsigned>(127 + 14 - min(e, 127)) << 23);
  *down = __uint_as_float(static_cast<unsigned>(127 - 14 + min(e, 127)) << 23);
}

// v = p0 + 2^-11 p1 with two f16 pieces (|v| < 2^16).  A NaN or Inf gives NaN.
__device__ __forceinline__ void split_pieces(float v, __half* p0, __half* p1) {
  *p0 = __float2half_rn(v);
  *p1 = __float2half_rn((v - __half2float(*p0)) * 2048.f);
}

// D = A B + C, A 16 x 16 and B 16 x 8 of f16, D and C fp32.
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint2 b) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b.x), "r"(b.y));
}

// One lane's part of a block: 16 columns of its four rows of both 16-row
// steps, and the columns' scale bytes.
struct RowSet {
  uint2 w[2][4];
  uint4 s;

  // Row row(step, i) of the block (255: none, read as zeros).  base points
  // at this lane's columns of the block's first row, scales at the block's.
  template <typename Row>
  __device__ __forceinline__ void load(const uint8_t* base, size_t row_bytes, const uint8_t* scales, bool any,
                                       Row row) {
#pragma unroll
    for (int step = 0; step < 2; ++step)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t r = row(step, i);
        w[step][i] = r < 32u ? __ldcs(reinterpret_cast<const uint2*>(base + r * row_bytes)) : make_uint2(0u, 0u);
      }
    s = any ? __ldg(reinterpret_cast<const uint4*>(scales)) : make_uint4(0u, 0u, 0u, 0u);
  }
};

// The A operands of one 8-column half: E pairs the even columns of two rows,
// O the odd ones (column 2 q in byte q).
__device__ __forceinline__ void pair_rows(uint32_t r0, uint32_t r1, uint32_t* even, uint32_t* odd) {
  constexpr uint32_t kLow = 0x0f0f0f0fu;
  *even = (r0 & kLow) | ((r1 << 4) & ~kLow);
  *odd = ((r0 >> 4) & kLow) | (r1 & ~kLow);
}

// acc[n][q][h] += (block product of token 4 n + t and column 2 q + h of the
// lane's 16): one or two 16-row steps into fresh accumulators, then the
// scales.  b[step][n] is the lane's B operand, sx[n] its token's scale.
template <int NT>
__device__ __forceinline__ void block_product(const RowSet& rs, bool two, const uint2 (&b)[2][NT],
                                              const float (&sx)[NT], float (&acc)[NT][8][2]) {
  const uint32_t sw[4] = {rs.s.x, rs.s.y, rs.s.z, rs.s.w};
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    // [step][e01, o01, e23, o23][column pair]
    uint32_t a[2][4][4];
#pragma unroll
    for (int step = 0; step < 2; ++step) {
      if (step == 1 && !two) break;
      uint32_t r[4], e01, o01, e23, o23;
#pragma unroll
      for (int i = 0; i < 4; ++i) r[i] = half == 0 ? rs.w[step][i].x : rs.w[step][i].y;
      pair_rows(r[0], r[1], &e01, &o01);
      pair_rows(r[2], r[3], &e23, &o23);
      e2m1_to_f16(e01, a[step][0]);
      e2m1_to_f16(o01, a[step][1]);
      e2m1_to_f16(e23, a[step][2]);
      e2m1_to_f16(o23, a[step][3]);
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      float d[NT][4];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        d[n][0] = d[n][1] = d[n][2] = d[n][3] = 0.f;
        mma_f16(d[n], a[0][0][q], a[0][1][q], a[0][2][q], a[0][3][q], b[0][n]);
      }
      if (two) {
#pragma unroll
        for (int n = 0; n < NT; ++n) mma_f16(d[n], a[1][0][q], a[1][1][q], a[1][2][q], a[1][3][q], b[1][n]);
      }
      float s0, s1;
      scale_pair(q & 1 ? sw[2 * half + q / 2] >> 16 : sw[2 * half + q / 2] & 0xffffu, &s0, &s1);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        // d[0], d[1]: the two pieces of column 2 q; d[2], d[3] of column 2 q + 1
        acc[n][4 * half + q][0] += fmaf(d[n][1], 0x1p-11f, d[n][0]) * sx[n] * s0;
        acc[n][4 * half + q][1] += fmaf(d[n][3], 0x1p-11f, d[n][2]) * sx[n] * s1;
      }
    }
  }
}

// The B operands of up to 4 nt tokens over all their blocks, in global memory:
// pieces [block][step][token / 4][2 (token % 4) + piece][16] f16, scales
// [block][4 nt], and a word per block and token of which rows are not zero.
struct Operand {
  __half* piece = nullptr;
  float* sx = nullptr;
  unsigned* mask = nullptr;
  int nt = 0;

  // Lane `lane` of a whole warp holds value v of row `lane` of a block of
  // token m; the warp writes its operand.
  __device__ __forceinline__ void put(int block, int m, float v, int lane) const {
    const unsigned top = __reduce_max_sync(0xffffffffu, __float_as_uint(v) & 0x7fffffffu);
    const unsigned kept = __ballot_sync(0xffffffffu, v != 0.f);
    float up, down;
    piece_scale(top, &up, &down);
    __half p0, p1;
    split_pieces(v * up, &p0, &p1);
    __half* at = piece + ((((size_t)block * 2 + (lane >> 4)) * nt + (m >> 2)) * 8 + (m & 3) * 2) * 16 + (lane & 15);
    at[0] = p0;
    at[16] = p1;
    if (lane == 0) {
      sx[(size_t)block * 4 * nt + m] = down;
      mask[(size_t)block * 4 * nt + m] = kept;
    }
  }
};

}  // namespace mx4
}  // namespace larosa
