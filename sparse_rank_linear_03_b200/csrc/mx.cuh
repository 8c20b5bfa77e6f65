// Microscaled blocks: 32 consecutive values of a row share one power of two.
//
//   scale byte e (ue8m0): 2^(e − 127); 255 marks a block that stands for NaN.
//   e2m1: 4-bit floats {0, .5, 1, 1.5, 2, 3, 4, 6} and their negatives (bit 3 of
//         the code is the sign), value = q · 2^(e−127); element 2i of a row is
//         the low half of byte i.
//   int8: value = q · 2^(e−127) / 64, −127 ≤ q ≤ 127.
//
// Codes are row-major with whole blocks per row (16 or 32 bytes each); the scale
// bytes of a row are padded to a multiple of 16, so that both can be read with
// 16-byte loads and copied as tiles.  Padding holds zeros.
#pragma once

#include "common.cuh"
#include "hsl.h"

namespace hsl {
namespace mx {

constexpr int kBlock = 32;

__host__ __device__ constexpr int64_t blocks(int64_t cols) { return (cols + kBlock - 1) / kBlock; }
__host__ __device__ constexpr int64_t code_pitch(int64_t cols, bool int8) {
  return blocks(cols) * (int8 ? 32 : 16);
}
__host__ __device__ constexpr int64_t scale_pitch(int64_t cols) {
  return (blocks(cols) + 15) / 16 * 16;
}

// 2^(e − 127) in fp32: every ue8m0 power is an fp32 value (2^−127 a subnormal).
__device__ __forceinline__ float scale_f32(uint32_t e) {
  return __uint_as_float(e == 255 ? 0x7FC00000u : e == 0 ? 0x00400000u : e << 23);
}

// Two e2m1 codes of a byte's low and high half, widened exactly.
__device__ __forceinline__ float e2m1_f32(uint32_t code) {
  const uint32_t mag = code & 7u;
  // 0 → 0, 1 → 0.5; otherwise exponent (code >> 1) − 1, mantissa bit (code & 1)
  const uint32_t bits = mag < 2u ? (mag ? 0x3F000000u : 0u) : 0x3F000000u + (mag << 22);
  return __uint_as_float(bits | ((code & 8u) << 28));
}

__device__ __forceinline__ uint32_t mul_bf2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t sub_bf2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// 2^(e − 127) as a pair of bf16 (2^−127 is a subnormal; 255 stands for NaN).
__device__ __forceinline__ uint32_t e2m1_scale(uint32_t e) {
  const uint32_t b = e == 255u ? 0x7FC0u : e == 0u ? 0x0040u : e << 7;
  return b | (b << 16);
}
// 2^(e − 127) / 64 (down to the subnormal 2^−133).
__device__ __forceinline__ uint32_t int8_scale(uint32_t e) {
  const uint32_t b = e == 255u ? 0x7FC0u : e > 6u ? (e - 6u) << 7 : 1u << e;
  return b | (b << 16);
}

// Eight e2m1 codes (one word) → eight bf16, exactly.  The high and the low byte of
// the eight magnitudes are looked up by byte permutes (a code's three low bits are
// the selector), the sign bits gathered by a third.
__device__ __forceinline__ uint4 widen_e2m1(uint32_t w, uint32_t scale) {
  const uint32_t mag = w & 0x77777777u, w4 = w << 4;
  uint32_t hi = __byte_perm(0x3F3F3F00u, 0x40404040u, mag);
  uint32_t lo = __byte_perm(0xC0800000u, 0xC0804000u, mag);
  hi |= __byte_perm(w4, w, 0x5140) & 0x80808080u;
  uint4 v;
  v.x = mul_bf2(__byte_perm(lo, hi, 0x5140), scale);
  v.y = mul_bf2(__byte_perm(lo, hi, 0x7362), scale);
  const uint32_t mag2 = mag >> 16;
  hi = __byte_perm(0x3F3F3F00u, 0x40404040u, mag2);
  lo = __byte_perm(0xC0800000u, 0xC0804000u, mag2);
  hi |= __byte_perm(w4, w, 0x7362) & 0x80808080u;
  v.z = mul_bf2(__byte_perm(lo, hi, 0x5140), scale);
  v.w = mul_bf2(__byte_perm(lo, hi, 0x7362), scale);
  return v;
}
// Four int8 (one word) → four bf16, exactly: 128 + (low 7 bits) is 0x4300 | bits, from
// which 128 (0x4300) or, for a negative value, 256 (0x4380) is taken away.
__device__ __forceinline__ uint2 widen_int8(uint32_t w, uint32_t scale) {
  const uint32_t m = w & 0x7F7F7F7Fu, n = w & 0x80808080u;
  uint2 v;
  v.x = mul_bf2(sub_bf2(__byte_perm(m, 0x43434343u, 0x4140), __byte_perm(n, 0x43434343u, 0x4140)), scale);
  v.y = mul_bf2(sub_bf2(__byte_perm(m, 0x43434343u, 0x4342), __byte_perm(n, 0x43434343u, 0x4342)), scale);
  return v;
}

// For rows that start anywhere: w becomes the NW words that start at byte `sh` (0 to 15) of its NW + 4, with the
// shift in binary steps so that no register is addressed by a variable.
template <int NW>
__device__ __forceinline__ void shift_bytes(uint32_t (&w)[NW + 4], uint32_t sh) {
#pragma unroll
  for (int i = 0; i < NW + 2; ++i) w[i] = sh & 8 ? w[i + 2] : w[i];
#pragma unroll
  for (int i = 0; i < NW + 1; ++i) w[i] = sh & 4 ? w[i + 1] : w[i];
#pragma unroll
  for (int i = 0; i < NW; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], (sh & 3) * 8);
}

}  // namespace mx
}  // namespace hsl
