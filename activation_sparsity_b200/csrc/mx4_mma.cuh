// Products of a few tokens with rows of a 4-bit (MX4) weight on mma.sync,
// shared by the sparse linear and the expert layer: see mx4_rows.cu for the
// arithmetic.  A warp multiplies blocks of 32 rows by 128 columns; lane
// (g, t) = (lane / 4, lane % 4) holds the columns 16 g .. 16 g + 15 of the
// rows 4 t .. 4 t + 3 of a 16-row step.
//
// Two layouts of the eight columns of a B operand: up to four tokens, column
// 2 token + piece (both pieces in one MMA); more tokens, eight tokens of one
// piece, an MMA per piece, so that a lane's two accumulator columns are two
// tokens and the scaling runs on pairs (fma.rn.f32x2).
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

// v = p0 + 2^-11 p1 with two f16 pieces (|v| < 2^16), to 2^-23 of v or 2^-36.  A
// NaN or Inf gives NaN.
__device__ __forceinline__ void split_pieces(float v, __half* p0, __half* p1) {
  *p0 = __float2half_rn(v);
  *p1 = __float2half_rn((v - __half2float(*p0)) * 2048.f);
}

// D = A B, or D += A B, with A 16 x 16 and B 16 x 8 of f16, D fp32.
__device__ __forceinline__ void mma_f16(float (&d)[4], bool fresh, uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint2 b) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %11, %12, %13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b.x), "r"(b.y), "f"(fresh ? 0.f : d[0]), "f"(fresh ? 0.f : d[1]),
        "f"(fresh ? 0.f : d[2]), "f"(fresh ? 0.f : d[3]));
}
// The same with a reduction of 8: A 16 x 8, B 8 x 8.
__device__ __forceinline__ void mma_f16_k8(float (&d)[4], bool fresh, uint32_t a0, uint32_t a1, uint32_t b) {
  asm("mma.sync.aligned.m16n8k8.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5}, {%6}, {%7, %8, %9, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(b), "f"(fresh ? 0.f : d[0]), "f"(fresh ? 0.f : d[1]), "f"(fresh ? 0.f : d[2]),
        "f"(fresh ? 0.f : d[3]));
}

// A block of 32 rows by 128 columns in shared memory, as a warp's copies
// leave it: the rows of both steps (position 16 step + 4 i + t holds row i of
// the lanes t, so that a warp reads 256 contiguous bytes for each i) and the
// columns' scale bytes.
struct __align__(16) Tile {
  uint8_t row[32][64];
  uint8_t scale[128];
};

// One lane's part of a tile: 16 columns of its rows of both steps (four of
// a 16-row step, two of an 8-row one), and the columns' scale bytes.
struct RowSet {
  uint2 w[2][4];
  uint4 s;

  template <int R0, int R1>
  __device__ __forceinline__ void read(const Tile& tile, int g, int t) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i < R0) w[0][i] = *reinterpret_cast<const uint2*>(&tile.row[4 * i + t][8 * g]);
      if (i < R1) w[1][i] = *reinterpret_cast<const uint2*>(&tile.row[16 + 4 * i + t][8 * g]);
    }
    s = *reinterpret_cast<const uint4*>(&tile.scale[16 * g]);
  }
};

// Asynchronous copies of 16 bytes to shared memory, through L2 only
// (weights) or also L1 (operands that other warps of the SM read too).
__device__ __forceinline__ void copy16_l2(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void copy16_l1(void* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Waits until at most `pending` of this thread's latest groups are in flight.
template <int pending>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(pending) : "memory");
}

// The A operands of one 8-column half: E pairs the even columns of two rows,
// O the odd ones (column 2 q in byte q).
__device__ __forceinline__ void pair_rows(uint32_t r0, uint32_t r1, uint32_t* even, uint32_t* odd) {
  constexpr uint32_t kLow = 0x0f0f0f0fu;
  *even = (r0 & kLow) | ((r1 << 4) & ~kLow);
  *odd = ((r0 >> 4) & kLow) | (r1 & ~kLow);
}

// Column pair q of one 8-column half: the steps' products into a fresh
// accumulator, then the scales into acc.  w[step]: e01, o01, e23, o23.
template <int NT, int R0, int R1, int q>
__device__ __forceinline__ void column_pair(const uint32_t (&w)[2][4], uint32_t scales, const uint2 (&b)[2][NT],
                                            const float (&sx)[NT], float (&acc)[NT][8][2], int at) {
  float d[NT][4];
#pragma unroll
  for (int step = 0; step < 2; ++step) {
    const int R = step == 0 ? R0 : R1;
    if (R == 0) continue;
    const uint32_t a0 = e2m1_to_f16<q>(w[step][0]), a1 = e2m1_to_f16<q>(w[step][1]);
    if (R == 4) {
      const uint32_t a2 = e2m1_to_f16<q>(w[step][2]), a3 = e2m1_to_f16<q>(w[step][3]);
#pragma unroll
      for (int n = 0; n < NT; ++n) mma_f16(d[n], step == 0, a0, a1, a2, a3, b[step][n]);
    } else {
#pragma unroll
      for (int n = 0; n < NT; ++n) mma_f16_k8(d[n], step == 0, a0, a1, b[step][n].x);
    }
  }
  float s0, s1;
  scale_pair(q & 1 ? scales >> 16 : scales & 0xffffu, &s0, &s1);
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    // d[0], d[1]: the two pieces of column 2 q; d[2], d[3] of column 2 q + 1
    acc[n][at][0] += fmaf(d[n][1], 0x1p-11f, d[n][0]) * sx[n] * s0;
    acc[n][at][1] += fmaf(d[n][3], 0x1p-11f, d[n][2]) * sx[n] * s1;
  }
}

// acc[n][q][h] += (block product of token 4 n + t and column 2 q + h of the
// lane's 16): steps of R0 and R1 rows per lane (4: 16 rows, 2: 8 rows, 0:
// none) into fresh accumulators, then the scales.  b[step][n] is the lane's B
// operand (.x alone for an 8-row step), sx[n] its token's scale.
template <int NT, int R0, int R1>
__device__ __forceinline__ void block_product(const RowSet& rs, const uint2 (&b)[2][NT], const float (&sx)[NT],
                                              float (&acc)[NT][8][2]) {
  const uint32_t sw[4] = {rs.s.x, rs.s.y, rs.s.z, rs.s.w};
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    uint32_t w[2][4];
#pragma unroll
    for (int step = 0; step < 2; ++step) {
      const int R = step == 0 ? R0 : R1;
      if (R == 0) continue;
      uint32_t r[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < R) r[i] = half == 0 ? rs.w[step][i].x : rs.w[step][i].y;
      pair_rows(r[0], r[1], &w[step][0], &w[step][1]);
      if (R == 4) pair_rows(r[2], r[3], &w[step][2], &w[step][3]);
    }
    column_pair<NT, R0, R1, 0>(w, sw[2 * half], b, sx, acc, 4 * half);
    column_pair<NT, R0, R1, 1>(w, sw[2 * half], b, sx, acc, 4 * half + 1);
    column_pair<NT, R0, R1, 2>(w, sw[2 * half + 1], b, sx, acc, 4 * half + 2);
    column_pair<NT, R0, R1, 3>(w, sw[2 * half + 1], b, sx, acc, 4 * half + 3);
  }
}

// ---------------------------------------------------------------- eight tokens per operand

__device__ __forceinline__ unsigned long long pack2(float lo, float hi) {
  unsigned long long r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 unpack2(unsigned long long v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ unsigned long long fma2(unsigned long long a, unsigned long long b, unsigned long long c) {
  unsigned long long r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ unsigned long long mul2(unsigned long long a, unsigned long long b) {
  unsigned long long r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// Column pair q: see block_product8.
template <int O, int q>
__device__ __forceinline__ void column_pair8(const uint32_t (&w)[2][4], uint32_t scales, const uint2 (&b)[2][O][2],
                                             const unsigned long long (&sx)[O], unsigned long long (&acc)[O][16],
                                             int at) {
  const uint32_t a[2][4] = {
      {e2m1_to_f16<q>(w[0][0]), e2m1_to_f16<q>(w[0][1]), e2m1_to_f16<q>(w[0][2]), e2m1_to_f16<q>(w[0][3])},
      {e2m1_to_f16<q>(w[1][0]), e2m1_to_f16<q>(w[1][1]), e2m1_to_f16<q>(w[1][2]), e2m1_to_f16<q>(w[1][3])}};
  float s0, s1;
  scale_pair(q & 1 ? scales >> 16 : scales & 0xffffu, &s0, &s1);
  const unsigned long long ss0 = pack2(s0, s0), ss1 = pack2(s1, s1), low = pack2(0x1p-11f, 0x1p-11f);
#pragma unroll
  for (int o = 0; o < O; ++o) {
    float d0[4], d1[4];
    mma_f16(d0, true, a[0][0], a[0][1], a[0][2], a[0][3], b[0][o][0]);
    mma_f16(d1, true, a[0][0], a[0][1], a[0][2], a[0][3], b[0][o][1]);
    mma_f16(d0, false, a[1][0], a[1][1], a[1][2], a[1][3], b[1][o][0]);
    mma_f16(d1, false, a[1][0], a[1][1], a[1][2], a[1][3], b[1][o][1]);
    const unsigned long long v0 = fma2(pack2(d1[0], d1[1]), low, pack2(d0[0], d0[1]));
    const unsigned long long v1 = fma2(pack2(d1[2], d1[3]), low, pack2(d0[2], d0[3]));
    acc[o][at] = fma2(mul2(v0, sx[o]), ss0, acc[o][at]);
    acc[o][at + 1] = fma2(mul2(v1, sx[o]), ss1, acc[o][at + 1]);
  }
}

// acc[o][c] += (block product of the tokens 8 o + 2 t and 8 o + 2 t + 1 and
// column c of the lane's 16), all 32 rows.  b[step][o][piece]: B operands;
// sx[o]: the two tokens' scales.
template <int O>
__device__ __forceinline__ void block_product8(const RowSet& rs, const uint2 (&b)[2][O][2],
                                               const unsigned long long (&sx)[O], unsigned long long (&acc)[O][16]) {
  const uint32_t sw[4] = {rs.s.x, rs.s.y, rs.s.z, rs.s.w};
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    uint32_t w[2][4];
#pragma unroll
    for (int step = 0; step < 2; ++step) {
      uint32_t r[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) r[i] = half == 0 ? rs.w[step][i].x : rs.w[step][i].y;
      pair_rows(r[0], r[1], &w[step][0], &w[step][1]);
      pair_rows(r[2], r[3], &w[step][2], &w[step][3]);
    }
    column_pair8<O, 0>(w, sw[2 * half], b, sx, acc, 8 * half);
    column_pair8<O, 1>(w, sw[2 * half], b, sx, acc, 8 * half + 2);
    column_pair8<O, 2>(w, sw[2 * half + 1], b, sx, acc, 8 * half + 4);
    column_pair8<O, 3>(w, sw[2 * half + 1], b, sx, acc, 8 * half + 6);
  }
}

// ---------------------------------------------------------------- copies of whole blocks

// A warp's copies of 32-row blocks `stride` blocks apart, 128 columns each,
// into a ring of tiles.  A lane brings 16 bytes of four rows (tile positions
// lane / 4 + 8 j), the first eight lanes also 16 scale bytes.
struct BlockCopies {
  const uint8_t* rows;    // this lane's bytes of the next block's first row
  const uint8_t* scales;  // and of its scales
  size_t row_step, scale_step;
  uint32_t off[4];

  // Columns [c0, c0 + width) of a matrix of ld columns from block `block` on;
  // columns past the width name the last ones.
  __device__ __forceinline__ void start(const uint8_t* codes, const uint8_t* all_scales, int ld, int c0, int width,
                                        int block, int stride, int lane) {
    const uint32_t row_bytes = (uint32_t)ld / 2;
    rows = codes + (size_t)block * kBlock * row_bytes + c0 / 2 + min(16 * (lane & 3), width / 2 - 16);
    scales = all_scales + (size_t)block * ld + c0 + min(16 * lane, width - 16);
    row_step = (size_t)stride * kBlock * row_bytes;
    scale_step = (size_t)stride * ld;
#pragma unroll
    for (int j = 0; j < 4; ++j) off[j] = row_of(8 * j + (lane >> 2)) * row_bytes;
  }
  // Row of the block at a tile position.
  static __device__ __forceinline__ uint32_t row_of(int pos) {
    return (uint32_t)((pos & 16) + (pos & 3) * 4 + ((pos >> 2) & 3));
  }
  // Copies the next block and moves on; commits a group.
  __device__ __forceinline__ void next(Tile& tile, int lane) {
#pragma unroll
    for (int j = 0; j < 4; ++j) copy16_l2(&tile.row[8 * j + (lane >> 2)][16 * (lane & 3)], rows + off[j]);
    if (lane < 8) copy16_l2(&tile.scale[16 * lane], scales);
    rows += row_step;
    scales += scale_step;
  }
};

// The B operands of up to 8 octets tokens over all their blocks, in global memory:
// pieces [block][step][token / 8][piece][token % 8][16] f16, scales
// [block][8 octets], and a word per block and token of which rows are not
// zero.
struct Operand {
  __half* piece = nullptr;
  float* sx = nullptr;
  unsigned* mask = nullptr;
  int octets = 0;

  // Lane `lane` of a whole warp holds value v of row `lane` of a block of
  // token m; the warp writes its operand.
  __device__ __forceinline__ void put(int block, int m, float v, int lane) const {
    const unsigned top = __reduce_max_sync(0xffffffffu, __float_as_uint(v) & 0x7fffffffu);
    const unsigned kept = __ballot_sync(0xffffffffu, v != 0.f);
    float up, down;
    piece_scale(top, &up, &down);
    __half p0, p1;
    split_pieces(v * up, &p0, &p1);
    __half* at = piece + ((((size_t)block * 2 + (lane >> 4)) * octets + (m >> 3)) * 16 + (m & 7)) * 16 + (lane & 15);
    at[0] = p0;
    at[128] = p1;
    if (lane == 0) {
      sx[(size_t)block * 8 * octets + m] = down;
      mask[(size_t)block * 8 * octets + m] = kept;
    }
  }
};

}  // namespace mx4
}  // namespace larosa
