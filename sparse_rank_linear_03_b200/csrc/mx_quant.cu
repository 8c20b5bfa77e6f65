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
// Bound by HBM: 2 + 0.53 (bf16, e2m1) to 4 + 1.03 bytes per element and no reuse; to keep
// up, an element may cost about five instructions.  A thread takes half a block (two
// or four 16-byte loads, one store of 8 or 16 bytes), shares the block's maximum with its
// neighbour by one shuffle, and takes the maximum of bf16 input two values at a
// time.  Two half blocks per thread are in flight.
#include <cuda_fp4.h>

#include "common.cuh"
#include "internal.h"
#include "mx.cuh"

namespace hsl {
namespace {

constexpr int Q_THREADS = 256;
constexpr int Q_UNROLL = 2;  // half blocks per thread, loads issued before the arithmetic

// u / d and u % d for 32-bit u by a multiplication: d's magic number is ceil(2^(32 + s) / d) − 2^32
// with s = ceil(log2 d) (Granlund and Montgomery, "Division by Invariant Integers using
// Multiplication", 1994).
struct FastDiv {
  uint32_t d, magic, shift;
};
FastDiv fast_div(uint32_t d) {
  uint32_t s = 0;
  while ((uint64_t(1) << s) < d) ++s;
  const uint64_t magic = ((uint64_t(1) << 32) * ((uint64_t(1) << s) - d)) / d + 1;
  return {d, uint32_t(magic), s};
}
__device__ __forceinline__ uint32_t div_by(uint32_t u, const FastDiv& f) {
  const uint32_t h = __umulhi(u, f.magic);
  return f.shift ? (((u - h) >> 1) + h) >> (f.shift - 1) : u;
}

// Row and half block in the row of half block u, hpr = 2 · blocks(cols) per row; 32-bit arithmetic
// where the numbers allow it.
__device__ __forceinline__ void locate(int64_t u, const FastDiv& hpr, bool small, int64_t& row, uint32_t& at) {
  if (small) {
    const uint32_t r = div_by(uint32_t(u), hpr);
    row = r;
    at = uint32_t(u) - r * hpr.d;
  } else {
    row = u / hpr.d;
    at = uint32_t(u - row * hpr.d);
  }
}

// Sixteen values as they are stored: 2 or 4 registers of 16 bytes.
template <typename T>
struct Half16 {
  uint4 q[sizeof(T)];
};
template <typename T>
__device__ __forceinline__ void load16(const T* p, Half16<T>& v) {
#pragma unroll
  for (int j = 0; j < int(sizeof(T)); ++j) v.q[j] = ld_stream16(reinterpret_cast<const uint4*>(p) + j);
}

// Largest |x| as fp32 bits.
__device__ __forceinline__ uint32_t top_bits(const Half16<float>& v) {
  uint32_t top = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    top = max(max(max(top, v.q[j].x & 0x7FFFFFFFu), max(v.q[j].y & 0x7FFFFFFFu, v.q[j].z & 0x7FFFFFFFu)),
              v.q[j].w & 0x7FFFFFFFu);
  return top;
}
__device__ __forceinline__ uint32_t top_bits(const Half16<__nv_bfloat16>& v) {
  uint32_t t = 0;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    t = __vmaxu2(t, __vmaxu2(v.q[j].x & 0x7FFF7FFFu, v.q[j].y & 0x7FFF7FFFu));
    t = __vmaxu2(t, __vmaxu2(v.q[j].z & 0x7FFF7FFFu, v.q[j].w & 0x7FFF7FFFu));
  }
  return max(t << 16, t & 0xFFFF0000u);
}
__device__ __forceinline__ void to_f32(const Half16<float>& v, float (&f)[16]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    f[4 * j] = __uint_as_float(v.q[j].x); f[4 * j + 1] = __uint_as_float(v.q[j].y);
    f[4 * j + 2] = __uint_as_float(v.q[j].z); f[4 * j + 3] = __uint_as_float(v.q[j].w);
  }
}
__device__ __forceinline__ void to_f32(const Half16<__nv_bfloat16>& v, float (&f)[16]) {
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    f[8 * j] = bf_lo(v.q[j].x); f[8 * j + 1] = bf_hi(v.q[j].x);
    f[8 * j + 2] = bf_lo(v.q[j].y); f[8 * j + 3] = bf_hi(v.q[j].y);
    f[8 * j + 4] = bf_lo(v.q[j].z); f[8 * j + 5] = bf_hi(v.q[j].z);
    f[8 * j + 6] = bf_lo(v.q[j].w); f[8 * j + 7] = bf_hi(v.q[j].w);
  }
}

// Four values → four int8 codes of 1/64: x / s first (64 / s alone may overflow), then a number whose
// last bits are the rounded integer.
__device__ __forceinline__ uint32_t int8_codes(float a, float b, float c, float d, float inv) {
  const float x[4] = {a * inv, b * inv, c * inv, d * inv};
  uint32_t w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    // 64 x is at most 128 in size; adding 1.5 · 2^23 rounds it to an integer (ties to even)
    const float r = fminf(fmaxf(fmaf(x[j], 64.f, 12582912.f), 12582912.f - 127.f), 12582912.f + 127.f);
    w[j] = __float_as_uint(r);
  }
  return __byte_perm(__byte_perm(w[0], w[1], 0x0040), __byte_perm(w[2], w[3], 0x0040), 0x5410);
}

// kVec: every half block is whole and 16-byte aligned (cols % 16 == 0, aligned base).  Otherwise a whole half
// block is put together from the aligned pieces around it, as long as these lie inside X
// (22859 × 10275 bf16 to int8: 180 µs; value by value 236).
template <typename T, bool kInt8, bool kVec>
__global__ void __launch_bounds__(Q_THREADS)
    k_mx_quantize(const T* __restrict__ X, const T* end, int64_t halves, const FastDiv hpr, int64_t cols,
                  uint8_t* __restrict__ codes, uint8_t* __restrict__ scales, int64_t spitch) {
  const int64_t u0 = int64_t(blockIdx.x) * (Q_THREADS * Q_UNROLL) + threadIdx.x;
  const bool small = halves <= 0xFFFFFFFFll;
  Half16<T> v[Q_UNROLL];
  int64_t row[Q_UNROLL];
  uint32_t at[Q_UNROLL];
#pragma unroll
  for (int k = 0; k < Q_UNROLL; ++k) {
    const int64_t u = u0 + k * Q_THREADS;
#pragma unroll
    for (int j = 0; j < int(sizeof(T)); ++j) v[k].q[j] = make_uint4(0, 0, 0, 0);
    row[k] = -1;
    if (u >= halves) continue;
    locate(u, hpr, small, row[k], at[k]);
    const int64_t c = int64_t(at[k]) * 16;
    const T* p = X + row[k] * cols + c;
    if (kVec) {
      if (c < cols) load16<T>(p, v[k]);
    } else {
      using bits = typename VT<T>::bits_t;
      const bits* q = reinterpret_cast<const bits*>(p);
      constexpr int NV = sizeof(T);
      uint32_t w[4 * NV + 4] = {};
      const uint32_t sh = uint32_t(reinterpret_cast<uintptr_t>(p) & 15);
      const char* low = reinterpret_cast<const char*>(p) - sh;
      if (c + 16 <= cols && low >= reinterpret_cast<const char*>(X) &&
          low + 16 * NV + (sh ? 16 : 0) <= reinterpret_cast<const char*>(end)) {
#pragma unroll
        for (int j = 0; j < NV + 1; ++j) {
          if (j == NV && sh == 0) break;
          const uint4 x = __ldg(reinterpret_cast<const uint4*>(low) + j);
          w[4 * j] = x.x; w[4 * j + 1] = x.y; w[4 * j + 2] = x.z; w[4 * j + 3] = x.w;
        }
        mx::shift_bytes<4 * NV>(w, sh);
      } else {
#pragma unroll
      for (int j = 0; j < 16; ++j)
        if (c + j < cols) w[j * sizeof(T) / 4] |= uint32_t(q[j]) << (sizeof(T) == 2 ? (j & 1) * 16 : 0);
      }
#pragma unroll
      for (int j = 0; j < int(sizeof(T)); ++j)
        v[k].q[j] = make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
    }
  }
#pragma unroll
  for (int k = 0; k < Q_UNROLL; ++k) {
    // a block's halves are neighbouring lanes; lanes past the end take part with zeros
    uint32_t top = top_bits(v[k]);
    top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
    if (row[k] < 0) continue;
    const bool bad = top >= 0x7F800000u;
    const int ef = int(top >> 23) - (kInt8 ? 0 : 2);
    const uint32_t e = bad ? 255u : uint32_t(max(ef, 0));
    const float inv = __uint_as_float(e >= 254u ? 0x00400000u : (254u - e) << 23);  // 2^(127 − e)
    float f[16];
    to_f32(v[k], f);
    if (kInt8) {
      uint4 w = make_uint4(int8_codes(f[0], f[1], f[2], f[3], inv), int8_codes(f[4], f[5], f[6], f[7], inv),
                           int8_codes(f[8], f[9], f[10], f[11], inv),
                           int8_codes(f[12], f[13], f[14], f[15], inv));
      if (bad) w = make_uint4(0, 0, 0, 0);
      *reinterpret_cast<uint4*>(codes + row[k] * int64_t(hpr.d) * 16 + int64_t(at[k]) * 16) = w;
    } else {
      uint32_t w[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t b[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          b[j] = __nv_cvt_float2_to_fp4x2(make_float2(f[8 * h + 2 * j] * inv, f[8 * h + 2 * j + 1] * inv),
                                          __NV_E2M1, cudaRoundNearest);
        w[h] = __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
      }
      if (bad) w[0] = w[1] = 0u;
      *reinterpret_cast<uint2*>(codes + row[k] * int64_t(hpr.d) * 8 + int64_t(at[k]) * 8) =
          make_uint2(w[0], w[1]);
    }
    if ((at[k] & 1) == 0) {
      uint8_t* srow = scales + row[k] * spitch;
      const int64_t blk = at[k] >> 1;
      srow[blk] = uint8_t(e);
      if (at[k] + 2 == hpr.d)  // the row's last block also writes the padding
        for (int64_t b = blk + 1; b < spitch; ++b) srow[b] = 0;
    }
  }
}

// The same half blocks in the other direction, by way of bf16, which holds every value
// exactly (at most 7 significant bits, down to 2^−133; what is past its range is
// past fp32's).  (22859 × 10275 int8 to bf16: 172 µs; with value by value stores 1251.)
template <typename T, bool kInt8, bool kVec>
__global__ void __launch_bounds__(Q_THREADS)
    k_mx_dequantize(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales,
                    int64_t halves, const FastDiv hpr, int64_t cols, int64_t spitch, T* __restrict__ X) {
  const int64_t u0 = int64_t(blockIdx.x) * (Q_THREADS * Q_UNROLL) + threadIdx.x;
  const bool small = halves <= 0xFFFFFFFFll;
  uint4 w[Q_UNROLL];
  uint32_t e[Q_UNROLL], at[Q_UNROLL];
  int64_t row[Q_UNROLL];
#pragma unroll
  for (int k = 0; k < Q_UNROLL; ++k) {
    const int64_t u = u0 + k * Q_THREADS;
    row[k] = -1;
    w[k] = make_uint4(0, 0, 0, 0);
    e[k] = at[k] = 0;
    if (u >= halves) continue;
    locate(u, hpr, small, row[k], at[k]);
    if (kInt8) {
      w[k] = ld_stream16(codes + row[k] * int64_t(hpr.d) * 16 + int64_t(at[k]) * 16);
    } else {
      const uint2 q = ld_stream8(codes + row[k] * int64_t(hpr.d) * 8 + int64_t(at[k]) * 8);
      w[k] = make_uint4(q.x, q.y, 0, 0);
    }
    e[k] = __ldg(scales + row[k] * spitch + (at[k] >> 1));
  }
#pragma unroll
  for (int k = 0; k < Q_UNROLL; ++k) {
    uint4 v[2];
    if (kInt8) {
      const uint32_t s = mx::int8_scale(e[k]);
      const uint2 a = mx::widen_int8(w[k].x, s), b = mx::widen_int8(w[k].y, s);
      const uint2 c = mx::widen_int8(w[k].z, s), d = mx::widen_int8(w[k].w, s);
      v[0] = make_uint4(a.x, a.y, b.x, b.y);
      v[1] = make_uint4(c.x, c.y, d.x, d.y);
    } else {
      const uint32_t s = mx::e2m1_scale(e[k]);
      v[0] = mx::widen_e2m1(w[k].x, s);
      v[1] = mx::widen_e2m1(w[k].y, s);
    }
    if (sizeof(T) == 2 && kVec) {
      // the two lanes of a block swap, so that a store instruction writes whole 32-byte
      // sectors: first values 0-15 of the block, then 16-31
      const bool odd = at[k] & 1;
      const uint4 give = odd ? v[0] : v[1];
      uint4 got;
      got.x = __shfl_xor_sync(0xFFFFFFFFu, give.x, 1);
      got.y = __shfl_xor_sync(0xFFFFFFFFu, give.y, 1);
      got.z = __shfl_xor_sync(0xFFFFFFFFu, give.z, 1);
      got.w = __shfl_xor_sync(0xFFFFFFFFu, give.w, 1);
      if (row[k] < 0) continue;
      const int64_t c = int64_t(at[k] >> 1) * 32 + (odd ? 8 : 0);
      T* p = X + row[k] * cols + c;
      st_stream16(p, odd ? got : v[0]);
      if (c + 16 < cols) st_stream16(p + 16, odd ? v[1] : got);
      continue;
    }
    const uint32_t b[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w};
    const int64_t c = int64_t(at[k]) * 16;
    T* p = X + row[k] * cols + c;
    if (kVec) {
      if (row[k] >= 0 && c < cols) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          st_stream16(p + 4 * j, make_uint4(b[2 * j] << 16, b[2 * j] & 0xFFFF0000u, b[2 * j + 1] << 16,
                                            b[2 * j + 1] & 0xFFFF0000u));
      }
      continue;
    }
    // Any alignment: a lane stores the aligned pieces that begin in its half block, the last of them
    // with the first values of the next lane's; what no lane has whole (a row's ends, a
    // warp's) goes value by value.
    constexpr int NV = sizeof(T), kSize = sizeof(T);
    uint32_t w[4 * NV + 4];
#pragma unroll
    for (int j = 0; j < 4 * NV; ++j)
      w[j] = kSize == 2 ? b[j & 7] : (j & 1) ? b[(j >> 1) & 7] & 0xFFFF0000u : b[(j >> 1) & 7] << 16;
    uint32_t own[4 * NV];
#pragma unroll
    for (int j = 0; j < 4 * NV; ++j) own[j] = w[j];
#pragma unroll
    for (int j = 0; j < 4; ++j) w[4 * NV + j] = __shfl_down_sync(0xFFFFFFFFu, own[j], 1);
    if (row[k] < 0 || c >= cols) continue;
    const int lane = threadIdx.x & 31;
    const int mine = int(min(int64_t(16), cols - c));
    const int next = lane < 31 ? int(max(int64_t(0), min(int64_t(16), cols - c - 16))) : 0;
    const int d = int((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15);  // bytes before the first piece
    const bool before = lane > 0 && at[k] > 0 && mine * kSize >= d;  // the lane before stores those
    const bool after = d == 0 || (next > 0 && next * kSize >= d);    // the last piece is whole
    if (mine == 16) {
      mx::shift_bytes<4 * NV>(w, uint32_t(d));
      char* q = reinterpret_cast<char*>(p) + d;
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if (j + 1 < NV || after)
          st_stream16(q + 16 * j, make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]));
    }
    const int head = before ? 0 : min(d / kSize, mine);
    const int tail = mine < 16 ? d / kSize : after ? 16 : (d + 16 * (NV - 1)) / kSize;
    if (head == 0 && tail >= mine) continue;
    using bits = typename VT<T>::bits_t;
    bits* q = reinterpret_cast<bits*>(p);
#pragma unroll
    for (int j = 0; j < 16; ++j)
      if (j < head || (j >= tail && j < mine)) q[j] = bits(kSize == 2 ? own[(j >> 1) % (4 * NV)] >> ((j & 1) * 16) : own[j % (4 * NV)]);
  }
}

template <typename T, bool kInt8>
hsl_status quantize_t(const T* X, int64_t rows, int64_t cols, uint8_t* codes, uint8_t* scales,
                      cudaStream_t s) {
  const FastDiv hpr = fast_div(uint32_t(2 * mx::blocks(cols)));
  const int64_t halves = rows * int64_t(hpr.d);
  const unsigned grid = unsigned((halves + Q_THREADS * Q_UNROLL - 1) / (Q_THREADS * Q_UNROLL));
  const bool vec = cols % 16 == 0 && reinterpret_cast<uintptr_t>(X) % 16 == 0;
  note_launch();
  if (vec)
    k_mx_quantize<T, kInt8, true>
        <<<grid, Q_THREADS, 0, s>>>(X, X + rows * cols, halves, hpr, cols, codes, scales, mx::scale_pitch(cols));
  else
    k_mx_quantize<T, kInt8, false>
        <<<grid, Q_THREADS, 0, s>>>(X, X + rows * cols, halves, hpr, cols, codes, scales, mx::scale_pitch(cols));
  return cuda_fail(cudaGetLastError(), "block quantisation launch");
}

template <typename T, bool kInt8>
hsl_status dequantize_t(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols, T* X,
                        cudaStream_t s) {
  const FastDiv hpr = fast_div(uint32_t(2 * mx::blocks(cols)));
  const int64_t halves = rows * int64_t(hpr.d);
  const unsigned grid = unsigned((halves + Q_THREADS * Q_UNROLL - 1) / (Q_THREADS * Q_UNROLL));
  const bool vec = cols % 16 == 0 && reinterpret_cast<uintptr_t>(X) % 16 == 0;
  note_launch();
  if (vec)
    k_mx_dequantize<T, kInt8, true>
        <<<grid, Q_THREADS, 0, s>>>(codes, scales, halves, hpr, cols, mx::scale_pitch(cols), X);
  else
    k_mx_dequantize<T, kInt8, false>
        <<<grid, Q_THREADS, 0, s>>>(codes, scales, halves, hpr, cols, mx::scale_pitch(cols), X);
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
