// Microscaled 4-bit values (MX4): blocks of 32 that share one power of two.
//
// A block holds 32 consecutive values along the reduction of the product the
// matrix takes part in.  Its scale byte b stands for 2^(b - 127) (255: NaN);
// each value is a 4-bit float e2m1 (sign, two exponent bits, one mantissa
// bit: 0, 0.5, 1, 1.5, 2, 3, 4, 6) times that.  Two values share a byte, the
// even column in the low half.  The format is that of the Open Compute
// Project's microscaling specification (MXFP4).
//
// The conversions between packed e2m1 and f16, e2m1 and fp32, and scale
// bytes and bf16 are single instructions on sm_100a, and all exact in the
// directions used here except fp32 -> e2m1, which rounds to nearest even and
// saturates at 6.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace larosa {
namespace mx4 {

constexpr int kBlock = 32;

// Byte q of w, two e2m1 values, as an f16 pair (the low half of the byte in
// the low half of the pair).
template <int q>
__device__ __forceinline__ uint32_t e2m1_to_f16(uint32_t w) {
  uint32_t h;
  asm("{\n\t.reg .b8 b<4>;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b%2;\n\t}"
      : "=r"(h)
      : "r"(w), "n"(q));
  return h;
}

// Two fp32 values to one byte of e2m1 codes, `lo` in the low half; nearest
// even, saturated at 6.
__device__ __forceinline__ uint32_t f32_to_e2m1(float lo, float hi) {
  uint32_t r;
  asm("{\n\t.reg .b8 a;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.u32.u8 %0, a;\n\t}"
      : "=r"(r)
      : "f"(lo), "f"(hi));
  return r;
}

// Two scale bytes (the low 16 bits of s, low byte first) as fp32 powers of
// two; byte 0 is 2^-127 (a subnormal), byte 255 NaN.
__device__ __forceinline__ void scale_pair(uint32_t s, float* lo, float* hi) {
  uint32_t r;
  asm("{\n\t.reg .b16 a;\n\t"
      "cvt.u16.u32 a, %1;\n\t"
      "cvt.rn.bf16x2.ue8m0x2 %0, a;\n\t}"
      : "=r"(r)
      : "r"(s));
  *lo = __uint_as_float(r << 16);
  *hi = __uint_as_float(r & 0xffff0000u);
}

__device__ __forceinline__ float2 f16x2_to_f32(uint32_t h) {
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// The scale byte of a block whose largest magnitude has the fp32 bits `amax`
// (sign cleared): floor(log2 amax) - 2, so that amax / scale lies in [4, 8);
// not below 2^-127; an all-zero block takes 2^-127, a NaN or Inf 255.
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax) {
  const uint32_t e = amax >> 23;  // biased; 0 for subnormals
  return e == 255u ? 255u : e > 2u ? e - 2u : 0u;
}

// 2^(127 - b): the exact factor that divides a block by its scale 2^(b-127).
// b <= 252 for any block scale_byte() gives a finite scale.
__device__ __forceinline__ float scale_inverse(uint32_t b) { return __uint_as_float((254u - b) << 23); }

}  // namespace mx4
}  // namespace larosa
