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

// The fp32 value of element j of a row, given the row's codes and scales.
template <bool kInt8>
__device__ __forceinline__ float value(const uint8_t* codes, const uint8_t* scales, int64_t j) {
  const float s = scale_f32(scales[j >> 5]);
  if (kInt8) return float(reinterpret_cast<const int8_t*>(codes)[j]) * 0.015625f * s;
  return e2m1_f32((codes[j >> 1] >> ((j & 1) * 4)) & 15u) * s;
}

}  // namespace mx
}  // namespace hsl
