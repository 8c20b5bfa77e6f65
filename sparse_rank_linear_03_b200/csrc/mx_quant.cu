// Quantisation of a matrix into microscaled blocks of 32 along its rows, and back.
//
//   s = 2^(floor(log2 max|x|) − emax),  emax = 2 (e2m1) or 0 (int8)
//   q = x / s rounded to nearest even on the element's grid, saturating
//
// s is a power of two, so x / s and q · s are exact and the codes do not depend
// on how they are computed.  max|x| is taken as the largest bit pattern of |x|:
// its exponent field is the scale, and a NaN or an infinity shows as a pattern at
// or above the infinity's.
//
// Bound by HBM: 4 + 0.53 bytes (f32) or 2 + 0.53 bytes (bf16, e2m1) per element and
// no reuse.  A thread takes 8 elements of a block (one or two 16-byte loads, one 4-
// or 8-byte store), the four threads of a block share the maximum by two shuffles.
#include <cuda_fp4.h>

#include "common.cuh"
#include "internal.h"
#include "mx.cuh"

namespace hsl {
namespace {

constexpr int Q_THREADS = 256;
constexpr int Q_UNROLL = 4;  // units of 8 elements per thread, loads issued before the arithmetic

template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&v)[8]);
template <>
__device__ __forceinline__ void load8<float>(const float* p, float (&v)[8]) {
  const uint4 a = ld_stream16(p), b = ld_stream16(p + 4);
  v[0] = __uint_as_float(a.x); v[1] = __uint_as_float(a.y);
  v[2] = __uint_as_float(a.z); v[3] = __uint_as_float(a.w);
  v[4] = __uint_as_float(b.x); v[5] = __uint_as_float(b.y);
  v[6] = __uint_as_float(b.z); v[7] = __uint_as_float(b.w);
}
template <>
__device__ __forceinline__ void load8<__nv_bfloat16>(const __nv_bfloat16* p, float (&v)[8]) {
  const uint4 a = ld_stream16(p);
  v[0] = bf_lo(a.x); v[1] = bf_hi(a.x); v[2] = bf_lo(a.y); v[3] = bf_hi(a.y);
  v[4] = bf_lo(a.z); v[5] = bf_hi(a.z); v[6] = bf_lo(a.w); v[7] = bf_hi(a.w);
}

// Unit u is elements [8 (u mod upr), +8) of row u / upr, upr = 4 · blocks(cols) units per row.
// kVec: every unit is whole and 16-byte aligned (cols % 8 == 0, aligned base).
template <typename T, bool kInt8, bool kVec>
__global__ void __launch_bounds__(Q_THREADS)
    k_mx_quantize(const T* __restrict__ X, int64_t units, uint32_t upr, int64_t cols,
                  uint8_t* __restrict__ codes, uint8_t* __restrict__ scales, int64_t spitch) {
  const int64_t u0 = int64_t(blockIdx.x) * (Q_THREADS * Q_UNROLL) + threadIdx.x;
  float v[Q_UNROLL][8];
  int64_t row[Q_UNROLL];
  uint32_t in_row[Q_UNROLL];
#pragma unroll
  for (int k = 0; k < Q_UNROLL; ++k) {
    const int64_t u = u0 + k * Q_THREADS;
#pragma unroll
    for (int j = 0; j < 8; ++j) v[k][j] = 0.f;
    row[k] = -1;
    if (u >= units) continue;
    // 32-bit division where the numbers allow it: the 64-bit one costs more than the arithmetic
    if (units <= 0xFFFFFFFFll) {
      const uint32_t r = uint32_t(u) / upr;
      row[k] = r;
      in_row[k] = uint32_t(u) - r * upr;
    } else {
      row[k] = u / upr;
      in_row[k] = uint32_t(u - row[k] * upr);
    }
    const int64_t c = int64_t(in_row[k]) * 8;
    const T* p = X + row[k] * cols + c;
    if (kVec) {
      if (c < cols) load8<T>(p, v[k]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (c + j < cols) v[k][j] = VT<T>::f(p[j]);
    }
  }
#pragma unroll
  for (int k = 0; k < Q_UNROLL; ++k) {
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) top = max(top, __float_as_uint(v[k][j]) & 0x7FFFFFFFu);
    // units of a block are four neighbouring lanes (units and 4 are multiples of 4,
    // so a block never crosses a warp); lanes past the end take part with zeros
    top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
    top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
    if (row[k] < 0) continue;
    const bool bad = top >= 0x7F800000u;
    const int ef = int(top >> 23) - (kInt8 ? 0 : 2);
    const uint32_t e = bad ? 255u : uint32_t(max(ef, 0));
    const float inv = __uint_as_float(e >= 254u ? 0x00400000u : (254u - e) << 23);  // 2^(127 − e)
    const int64_t blk = in_row[k] >> 2;
    if (kInt8) {
      uint32_t w[2] = {0u, 0u};
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        // x / s first: 64 / s alone may overflow
        const int q = max(-127, min(127, __float2int_rn(v[k][j] * inv * 64.f)));
        w[j >> 2] |= uint32_t(q & 0xFF) << ((j & 3) * 8);
      }
      if (bad) w[0] = w[1] = 0u;
      *reinterpret_cast<uint2*>(codes + row[k] * int64_t(upr) * 8 + int64_t(in_row[k]) * 8) =
          make_uint2(w[0], w[1]);
    } else {
      uint32_t w = 0;
#pragma unroll
      for (int j = 0; j < 8; j += 2) {
        const __nv_fp4x2_storage_t q = __nv_cvt_float2_to_fp4x2(
            make_float2(v[k][j] * inv, v[k][j + 1] * inv), __NV_E2M1, cudaRoundNearest);
        w |= uint32_t(q) << (j * 4);
      }
      if (bad) w = 0u;
      *reinterpret_cast<uint32_t*>(codes + row[k] * int64_t(upr) * 4 + int64_t(in_row[k]) * 4) = w;
    }
    if ((in_row[k] & 3) == 0) {
      uint8_t* srow = scales + row[k] * spitch;
      srow[blk] = uint8_t(e);
      if (in_row[k] + 4 == upr)  // the row's last block also writes the padding
        for (int64_t b = blk + 1; b < spitch; ++b) srow[b] = 0;
    }
  }
}

template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&v)[8]);
template <>
__device__ __forceinline__ void store8<float>(float* p, const float (&v)[8]) {
  st_stream16(p, make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                            __float_as_uint(v[3])));
  st_stream16(p + 4, make_uint4(__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]),
                                __float_as_uint(v[7])));
}
__device__ __forceinline__ uint32_t bf_pack(float lo, float hi) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&p);
}
template <>
__device__ __forceinline__ void store8<__nv_bfloat16>(__nv_bfloat16* p, const float (&v)[8]) {
  st_stream16(p, make_uint4(bf_pack(v[0], v[1]), bf_pack(v[2], v[3]), bf_pack(v[4], v[5]),
                            bf_pack(v[6], v[7])));
}

// The same units in the other direction.  Every value is exact in fp32; bf16 holds
// it exactly too (at most 7 significant bits, down to 2^−133).
template <typename T, bool kInt8, bool kVec>
__global__ void __launch_bounds__(Q_THREADS)
    k_mx_dequantize(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales,
                    int64_t units, uint32_t upr, int64_t cols, int64_t spitch, T* __restrict__ X) {
  const int64_t u0 = int64_t(blockIdx.x) * (Q_THREADS * Q_UNROLL) + threadIdx.x;
  uint2 w[Q_UNROLL];
  uint32_t e[Q_UNROLL], in_row[Q_UNROLL];
  int64_t row[Q_UNROLL];
#pragma unroll
  for (int k = 0; k < Q_UNROLL; ++k) {
    const int64_t u = u0 + k * Q_THREADS;
    row[k] = -1;
    if (u >= units) continue;
    if (units <= 0xFFFFFFFFll) {
      const uint32_t r = uint32_t(u) / upr;
      row[k] = r;
      in_row[k] = uint32_t(u) - r * upr;
    } else {
      row[k] = u / upr;
      in_row[k] = uint32_t(u - row[k] * upr);
    }
    if (kInt8) {
      w[k] = ld_stream8(codes + row[k] * int64_t(upr) * 8 + int64_t(in_row[k]) * 8);
    } else {
      w[k].x = __ldg(reinterpret_cast<const uint32_t*>(codes + row[k] * int64_t(upr) * 4 +
                                                       int64_t(in_row[k]) * 4));
    }
    e[k] = __ldg(scales + row[k] * spitch + (in_row[k] >> 2));
  }
#pragma unroll
  for (int k = 0; k < Q_UNROLL; ++k) {
    if (row[k] < 0) continue;
    const float s = mx::scale_f32(e[k]);
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (kInt8) {
        const uint32_t word = j < 4 ? w[k].x : w[k].y;
        v[j] = float(int8_t(word >> ((j & 3) * 8))) * 0.015625f * s;
      } else {
        v[j] = mx::e2m1_f32((w[k].x >> (j * 4)) & 15u) * s;
      }
    }
    const int64_t c = int64_t(in_row[k]) * 8;
    T* p = X + row[k] * cols + c;
    if (kVec) {
      if (c < cols) store8<T>(p, v);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (c + j < cols) p[j] = VT<T>::from_f(v[j]);
    }
  }
}

template <typename T, bool kInt8>
hsl_status quantize_t(const T* X, int64_t rows, int64_t cols, uint8_t* codes, uint8_t* scales,
                      cudaStream_t s) {
  const uint32_t upr = uint32_t(4 * mx::blocks(cols));
  const int64_t units = rows * int64_t(upr);
  const unsigned grid = unsigned((units + Q_THREADS * Q_UNROLL - 1) / (Q_THREADS * Q_UNROLL));
  const bool vec = cols % 8 == 0 && reinterpret_cast<uintptr_t>(X) % 16 == 0;
  note_launch();
  if (vec)
    k_mx_quantize<T, kInt8, true>
        <<<grid, Q_THREADS, 0, s>>>(X, units, upr, cols, codes, scales, mx::scale_pitch(cols));
  else
    k_mx_quantize<T, kInt8, false>
        <<<grid, Q_THREADS, 0, s>>>(X, units, upr, cols, codes, scales, mx::scale_pitch(cols));
  return cuda_fail(cudaGetLastError(), "block quantisation launch");
}

template <typename T, bool kInt8>
hsl_status dequantize_t(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols, T* X,
                        cudaStream_t s) {
  const uint32_t upr = uint32_t(4 * mx::blocks(cols));
  const int64_t units = rows * int64_t(upr);
  const unsigned grid = unsigned((units + Q_THREADS * Q_UNROLL - 1) / (Q_THREADS * Q_UNROLL));
  const bool vec = cols % 8 == 0 && reinterpret_cast<uintptr_t>(X) % 16 == 0;
  note_launch();
  if (vec)
    k_mx_dequantize<T, kInt8, true>
        <<<grid, Q_THREADS, 0, s>>>(codes, scales, units, upr, cols, mx::scale_pitch(cols), X);
  else
    k_mx_dequantize<T, kInt8, false>
        <<<grid, Q_THREADS, 0, s>>>(codes, scales, units, upr, cols, mx::scale_pitch(cols), X);
  return cuda_fail(cudaGetLastError(), "block dequantisation launch");
}

}  // namespace

hsl_status mx_quantize_run(const void* X, hsl_dtype dtype, int64_t rows, int64_t cols, bool int8,
                           void* codes, void* scales, cudaStream_t s) {
  uint8_t* c = static_cast<uint8_t*>(codes);
  uint8_t* e = static_cast<uint8_t*>(scales);
  if (dtype == HSL_F32) {
    const float* x = static_cast<const float*>(X);
    return int8 ? quantize_t<float, true>(x, rows, cols, c, e, s)
                : quantize_t<float, false>(x, rows, cols, c, e, s);
  }
  const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(X);
  return int8 ? quantize_t<__nv_bfloat16, true>(x, rows, cols, c, e, s)
              : quantize_t<__nv_bfloat16, false>(x, rows, cols, c, e, s);
}

hsl_status mx_dequantize_run(const void* codes, const void* scales, int64_t rows, int64_t cols,
                             bool int8, void* X, hsl_dtype dtype, cudaStream_t s) {
  const uint8_t* c = static_cast<const uint8_t*>(codes);
  const uint8_t* e = static_cast<const uint8_t*>(scales);
  if (dtype == HSL_F32) {
    float* x = static_cast<float*>(X);
    return int8 ? dequantize_t<float, true>(c, e, rows, cols, x, s)
                : dequantize_t<float, false>(c, e, rows, cols, x, s);
  }
  __nv_bfloat16* x = static_cast<__nv_bfloat16*>(X);
  return int8 ? dequantize_t<__nv_bfloat16, true>(c, e, rows, cols, x, s)
              : dequantize_t<__nv_bfloat16, false>(c, e, rows, cols, x, s);
}

}  // namespace hsl
