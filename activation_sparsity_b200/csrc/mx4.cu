// Values to the microscaled 4-bit format and back (sm_100a): see mx4.cuh.
//
//   quantise     b = clamp(floor(log2 max|v|) - 2, -127, .), code = e2m1(v 2^-b)
//   dequantise   v = code 2^b
//
// over a row-major [rows x cols] matrix, blocks of 32 along a row (axis 1:
// activations, weights in torch.nn.Linear layout) or down a column (axis 0:
// row-major x . W weights, whose reduction runs down the rows).  The division
// by the scale is exact (a power of two), so a code is the correctly rounded
// one.
//
// Both directions are one pass over memory (2 or 4 bytes of value and 17/32
// of a byte of format per entry) and bound by HBM, so the kernels only have
// to keep enough wide loads in flight.  Every thread works on eight
// neighbouring entries of a row, the 4 bytes of codes they make:
//   axis 1  four lanes share a block; its maximum is two shuffles.  A thread
//           takes kU such groups, a whole grid apart, all loaded before the
//           first is used;
//   axis 0  a warp takes 32 rows x 64 columns, each thread 8 columns of 8
//           rows (rows 4 i + lane / 8): 128-byte row segments in, 32-byte
//           segments of codes out, the column maxima joined by two shuffles
//           across the four row lanes.
//
// Measured (B200, graph replay, from HBM, one direction after the other): 4096 x
// 22016 bf16, axis 0, 77.4 us (456 MB: 5.9 TB/s, the copy rate being 6.5), axis 1
// 75.7; the same in fp32, axis 0, 129.9 us (817 MB: 6.3 TB/s), axis 1 127.7; 777 x
// 11008 fp32, axis 1, 13.5 us (78 MB: 5.7 TB/s); one row of 4096, 2.1 us.
#include "common.cuh"
#include "internal.h"
#include "mx4.cuh"

namespace larosa {
namespace {

constexpr int kQThreads = 256;
constexpr int kU = 4;  // 8-entry groups per thread, axis 1

// Eight consecutive entries as fp32.
template <typename T>
struct Eight;
template <>
struct Eight<__nv_bfloat16> {
  uint4 u;
  __device__ __forceinline__ void load(const void* base, size_t i) {
    u = __ldcs(reinterpret_cast<const uint4*>(base) + i);
  }
  __device__ __forceinline__ void zero() { u = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ void store(void* base, size_t i, const float (&v)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const __nv_bfloat162 p = __floats2bfloat162_rn(v[2 * k], v[2 * k + 1]);  // exact: 2 mantissa bits
      w[k] = *reinterpret_cast<const uint32_t*>(&p);
    }
    reinterpret_cast<uint4*>(base)[i] = make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <>
struct Eight<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const void* base, size_t i) {
    a = __ldcs(reinterpret_cast<const float4*>(base) + 2 * i);
    b = __ldcs(reinterpret_cast<const float4*>(base) + 2 * i + 1);
  }
  __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
  static __device__ __forceinline__ void store(void* base, size_t i, const float (&v)[8]) {
    // 32 bytes at once where the matrix is aligned so: two 16-byte stores of a
    // warp leave every other half sector to each other (4.2 and 6.3 TB/s)
    float* at = static_cast<float*>(base) + 8 * i;
    if ((reinterpret_cast<uintptr_t>(base) & 31u) == 0) {
      asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(at), "f"(v[0]), "f"(v[1]),
                   "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
                   : "memory");
    } else {
      reinterpret_cast<float4*>(at)[0] = make_float4(v[0], v[1], v[2], v[3]);
      reinterpret_cast<float4*>(at)[1] = make_float4(v[4], v[5], v[6], v[7]);
    }
  }
};

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// Axis 1: `groups` groups of eight entries, four to a block.
template <typename T>
__global__ void __launch_bounds__(kQThreads)
    quantize_rows_kernel(const void* __restrict__ src, size_t groups, uint32_t* __restrict__ codes,
                         uint8_t* __restrict__ scales, int* dev_status) {
  pdl_wait();
  // the codes' readers wait for this grid before they read anything
  pdl_launch_dependents();
  const size_t stride = (size_t)gridDim.x * kQThreads;
  const size_t g0 = (size_t)blockIdx.x * kQThreads + threadIdx.x;
  Eight<T> e[kU];
#pragma unroll
  for (int u = 0; u < kU; ++u) {
    const size_t g = g0 + u * stride;
    if (g < groups)
      e[u].load(src, g);
    else
      e[u].zero();
  }
  bool bad = false;
#pragma unroll
  for (int u = 0; u < kU; ++u) {
    const size_t g = g0 + u * stride;
    float v[8];
    e[u].get(v);
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, abs_bits(v[i]));
    // a block's four lanes are all inside `groups` or all outside it
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
    const uint32_t b = mx4::scale_byte(m);
    uint32_t code = 0;
    if (b == 255u) {
      bad = true;
    } else {
      const float inv = mx4::scale_inverse(b);
#pragma unroll
      for (int i = 0; i < 4; ++i) code |= mx4::f32_to_e2m1(v[2 * i] * inv, v[2 * i + 1] * inv) << (8 * i);
    }
    if (g < groups) {
      codes[g] = code;
      if ((threadIdx.x & 3) == 0) scales[g >> 2] = static_cast<uint8_t>(b);
    }
  }
  if (__any_sync(0xffffffffu, bad) && (threadIdx.x & 31) == 0) report(dev_status, LAROSA_DEV_NONFINITE);
}

// The largest magnitudes of eight columns, as bits; those of bf16 in pairs, as
// they are loaded: one by one the maxima cost a fifth of the time of a pass
// over bf16 (axis 0: 51.6 and 40.2 us for 4096 x 22016).
template <typename T>
struct Tops;
template <>
struct Tops<__nv_bfloat16> {
  uint32_t m[4] = {0u, 0u, 0u, 0u};
  __device__ __forceinline__ void add(const Eight<__nv_bfloat16>& e) {
    const uint32_t w[4] = {e.u.x, e.u.y, e.u.z, e.u.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) m[k] = __vmaxu2(m[k], w[k] & 0x7fff7fffu);
  }
  __device__ __forceinline__ void join(int lanes) {
#pragma unroll
    for (int k = 0; k < 4; ++k) m[k] = __vmaxu2(m[k], __shfl_xor_sync(0xffffffffu, m[k], lanes));
  }
  __device__ __forceinline__ uint32_t bits(int k) const { return k & 1 ? m[k / 2] & 0xffff0000u : m[k / 2] << 16; }
};
template <>
struct Tops<float> {
  uint32_t m[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
  __device__ __forceinline__ void add(const Eight<float>& e) {
    float v[8];
    e.get(v);
#pragma unroll
    for (int k = 0; k < 8; ++k) m[k] = max(m[k], abs_bits(v[k]));
  }
  __device__ __forceinline__ void join(int lanes) {
#pragma unroll
    for (int k = 0; k < 8; ++k) m[k] = max(m[k], __shfl_xor_sync(0xffffffffu, m[k], lanes));
  }
  __device__ __forceinline__ uint32_t bits(int k) const { return m[k]; }
};

// Axis 0: warp tile 32 rows x 64 columns; cg = cols / 8 column groups.
template <typename T>
__global__ void __launch_bounds__(kQThreads, sizeof(T) == 2 ? 4 : 2)
    quantize_cols_kernel(const void* __restrict__ src, int row_blocks, int cg, uint32_t* __restrict__ codes,
                         uint8_t* __restrict__ scales, int* dev_status) {
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, rl = lane >> 3;
  const int tiles = (cg + 7) >> 3;
  const size_t n_tiles = (size_t)tiles * row_blocks;
  const size_t n_warps = (size_t)gridDim.x * (kQThreads / 32);
  bool bad = false;
  for (size_t t = (size_t)blockIdx.x * (kQThreads / 32) + (threadIdx.x >> 5); t < n_tiles; t += n_warps) {
    const int rb = static_cast<int>(t / tiles);
    const int c = static_cast<int>(t % tiles) * 8 + (lane & 7);
    const bool in = c < cg;
    const size_t at = ((size_t)rb * mx4::kBlock + rl) * cg + c;  // this thread's first group
    Eight<T> e[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (in)
        e[i].load(src, at + (size_t)(4 * i) * cg);
      else
        e[i].zero();
    }
    Tops<T> top;
#pragma unroll
    for (int i = 0; i < 8; ++i) top.add(e[i]);
    top.join(8);
    top.join(16);
    float inv[8];
    uint32_t sb[2] = {0, 0}, ok = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const uint32_t b = mx4::scale_byte(top.bits(k));
      sb[k >> 2] |= b << (8 * (k & 3));
      bad |= b == 255u;
      ok |= (b == 255u ? 0u : 0xfu) << (4 * k);
      inv[k] = b == 255u ? 0.f : mx4::scale_inverse(b);
    }
    if (in && rl == 0) reinterpret_cast<uint2*>(scales)[(size_t)rb * cg + c] = make_uint2(sb[0], sb[1]);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float v[8];
      e[i].get(v);
      uint32_t code = 0;
#pragma unroll
      for (int k = 0; k < 4; ++k)
        code |= mx4::f32_to_e2m1(v[2 * k] * inv[2 * k], v[2 * k + 1] * inv[2 * k + 1]) << (8 * k);
      if (in) codes[at + (size_t)(4 * i) * cg] = code & ok;  // a NaN block's codes are zero
    }
  }
  if (__any_sync(0xffffffffu, bad) && lane == 0) report(dev_status, LAROSA_DEV_NONFINITE);
}

// The eight values of a code word, not yet scaled.
__device__ __forceinline__ void code_values(uint32_t code, float (&v)[8]) {
  const uint32_t h[4] = {mx4::e2m1_to_f16<0>(code), mx4::e2m1_to_f16<1>(code), mx4::e2m1_to_f16<2>(code),
                         mx4::e2m1_to_f16<3>(code)};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = mx4::f16x2_to_f32(h[i]);
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}

// The values may be read as a weight by a kernel that starts loading weights
// before this grid has ended, so neither dequantising kernel lets the next
// one start early.
template <typename T>
__global__ void __launch_bounds__(kQThreads)
    dequantize_rows_kernel(const uint32_t* __restrict__ codes, const uint8_t* __restrict__ scales,
                           size_t groups, void* __restrict__ dst) {
  pdl_wait();
  const size_t stride = (size_t)gridDim.x * kQThreads;
  const size_t g0 = (size_t)blockIdx.x * kQThreads + threadIdx.x;
  uint32_t code[kU], b[kU];
#pragma unroll
  for (int u = 0; u < kU; ++u) {
    const size_t g = g0 + u * stride;
    code[u] = g < groups ? __ldcs(codes + g) : 0u;
    b[u] = g < groups ? __ldcs(scales + (g >> 2)) : 0u;
  }
#pragma unroll
  for (int u = 0; u < kU; ++u) {
    const size_t g = g0 + u * stride;
    if (g >= groups) break;
    float v[8], s, unused;
    code_values(code[u], v);
    mx4::scale_pair(b[u], &s, &unused);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] *= s;
    Eight<T>::store(dst, g, v);
  }
}

template <typename T>
__global__ void __launch_bounds__(kQThreads)
    dequantize_cols_kernel(const uint32_t* __restrict__ codes, const uint8_t* __restrict__ scales,
                           int row_blocks, int cg, void* __restrict__ dst) {
  pdl_wait();
  const int lane = threadIdx.x & 31, rl = lane >> 3;
  const int tiles = (cg + 7) >> 3;
  const size_t n_tiles = (size_t)tiles * row_blocks;
  const size_t n_warps = (size_t)gridDim.x * (kQThreads / 32);
  for (size_t t = (size_t)blockIdx.x * (kQThreads / 32) + (threadIdx.x >> 5); t < n_tiles; t += n_warps) {
    const int rb = static_cast<int>(t / tiles);
    const int c = static_cast<int>(t % tiles) * 8 + (lane & 7);
    if (c >= cg) continue;
    const size_t at = ((size_t)rb * mx4::kBlock + rl) * cg + c;
    uint32_t code[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) code[i] = __ldcs(codes + at + (size_t)(4 * i) * cg);
    const uint2 sb = reinterpret_cast<const uint2*>(scales)[(size_t)rb * cg + c];
    float s[8];
    mx4::scale_pair(sb.x & 0xffffu, &s[0], &s[1]);
    mx4::scale_pair(sb.x >> 16, &s[2], &s[3]);
    mx4::scale_pair(sb.y & 0xffffu, &s[4], &s[5]);
    mx4::scale_pair(sb.y >> 16, &s[6], &s[7]);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float v[8];
      code_values(code[i], v);
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] *= s[k];
      Eight<T>::store(dst, at + (size_t)(4 * i) * cg, v);
    }
  }
}

cudaLaunchConfig_t config(size_t blocks, cudaStream_t stream, cudaLaunchAttribute* attr) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks), 1, 1);
  cfg.blockDim = dim3(kQThreads, 1, 1);
  cfg.stream = stream;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cfg;
}

// Axis 1: kU groups per thread, but at least one CTA for every kQThreads
// groups up to 148 of them (a single token is latency, not bandwidth).
size_t row_blocks_of_grid(size_t groups) {
  const size_t one = (groups + kQThreads - 1) / kQThreads;
  const size_t full = (groups + (size_t)kQThreads * kU - 1) / ((size_t)kQThreads * kU);
  return full > 148 ? full : one < 148 ? one : 148;
}

size_t col_blocks_of_grid(int rows, int cols) {
  const size_t tiles = (size_t)((cols / 8 + 7) / 8) * (rows / mx4::kBlock);
  return (tiles + kQThreads / 32 - 1) / (kQThreads / 32);
}

}  // namespace

cudaError_t launch_mx4_quantize(const void* src, int rows, int cols, int axis, Elem elem, void* codes,
                                void* scales, int* dev_status, cudaStream_t stream) {
  cudaLaunchAttribute attr[1];
  uint32_t* c = static_cast<uint32_t*>(codes);
  uint8_t* s = static_cast<uint8_t*>(scales);
  if (axis == 1) {
    const size_t groups = (size_t)rows * (cols / 8);
    const cudaLaunchConfig_t cfg = config(row_blocks_of_grid(groups), stream, attr);
    return elem == Elem::BF16
               ? cudaLaunchKernelEx(&cfg, quantize_rows_kernel<__nv_bfloat16>, src, groups, c, s, dev_status)
               : cudaLaunchKernelEx(&cfg, quantize_rows_kernel<float>, src, groups, c, s, dev_status);
  }
  const cudaLaunchConfig_t cfg = config(col_blocks_of_grid(rows, cols), stream, attr);
  return elem == Elem::BF16 ? cudaLaunchKernelEx(&cfg, quantize_cols_kernel<__nv_bfloat16>, src,
                                                 rows / mx4::kBlock, cols / 8, c, s, dev_status)
                            : cudaLaunchKernelEx(&cfg, quantize_cols_kernel<float>, src, rows / mx4::kBlock,
                                                 cols / 8, c, s, dev_status);
}

cudaError_t launch_mx4_dequantize(const void* codes, const void* scales, int rows, int cols, int axis,
                                  Elem elem, void* dst, cudaStream_t stream) {
  cudaLaunchAttribute attr[1];
  const uint32_t* c = static_cast<const uint32_t*>(codes);
  const uint8_t* s = static_cast<const uint8_t*>(scales);
  if (axis == 1) {
    const size_t groups = (size_t)rows * (cols / 8);
    const cudaLaunchConfig_t cfg = config(row_blocks_of_grid(groups), stream, attr);
    return elem == Elem::BF16 ? cudaLaunchKernelEx(&cfg, dequantize_rows_kernel<__nv_bfloat16>, c, s, groups, dst)
                              : cudaLaunchKernelEx(&cfg, dequantize_rows_kernel<float>, c, s, groups, dst);
  }
  const cudaLaunchConfig_t cfg = config(col_blocks_of_grid(rows, cols), stream, attr);
  return elem == Elem::BF16 ? cudaLaunchKernelEx(&cfg, dequantize_cols_kernel<__nv_bfloat16>, c, s,
                                                 rows / mx4::kBlock, cols / 8, dst)
                            : cudaLaunchKernelEx(&cfg, dequantize_cols_kernel<float>, c, s, rows / mx4::kBlock,
                                                 cols / 8, dst);
}

}  // namespace larosa
