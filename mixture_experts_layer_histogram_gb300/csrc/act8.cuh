// Activations in 8 bits, in registers: blocks of 32 values along a row share one power of two (byte b stands for
// 2^(b - 127), 255 for NaN), codes are e4m3 (1 sign, 4 exponent and 3 mantissa bits, largest 448).
//
// The scale is the least 2^e with max|x| <= 448 2^e, not below 2^-127, so nothing saturates: with 448 = 1.75 * 2^8 that
// is e = (exponent of the maximum) - 8, and one more where its mantissa passes 1.75. Dividing by a power of two is
// exact, so codes depend on the input alone, and a code times its scale is exact in bf16 (4 significant bits) while it
// lies in the normal range.
#pragma once

#include "common.cuh"

namespace moe {
namespace act8 {

constexpr int kBlock = 32;   // values per scale

__host__ __device__ __forceinline__ int64_t blocks_of(int64_t K) { return (K + kBlock - 1) / kBlock; }

// The largest magnitude of three values; a NaN stays one
__device__ __forceinline__ float larger(float a, float b, float c) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// Scale byte of a block whose largest magnitude has the fp32 bits `amax` (sign clear). NaN bits are the largest
// integers, so an integer maximum carries a NaN through, and a block that is not finite gets 255.
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax) {
  if (amax >= 0x7f800000u) return 255u;
  const int e = (int)((amax + 0x1fffffu) >> 23) - 8;   // a mantissa above 0.75 carries into the exponent
  return e > 0 ? (uint32_t)e : 0u;
}
// 1 / scale as fp32 (0 for a NaN block: its codes are zeros)
__device__ __forceinline__ float inv_scale(uint32_t byte) { return __uint_as_float(byte == 255u ? 0u : (254u - byte) << 23); }
// The scale as fp32 (NaN for 255)
__device__ __forceinline__ float scale_value(uint32_t byte) {
  return __uint_as_float(byte == 255u ? 0x7fc00000u : (byte == 0 ? 0x00400000u : byte << 23));
}

// Four values (already divided by their scale) to four codes, the first in the low byte; round to nearest even.
__device__ __forceinline__ uint32_t pack4(float v0, float v1, float v2, float v3) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
      "mov.b32 %0, {lo, hi};\n\t}"
      : "=r"(r)
      : "f"(v0), "f"(v1), "f"(v2), "f"(v3));
  return r;
}
// Four codes to four values (before their scale)
__device__ __forceinline__ void unpack4(uint32_t q, float *v) {
  asm("{\n\t.reg .b16 lo, hi, a, b, c, d;\n\t.reg .b32 x, y;\n\t"
      "mov.b32 {lo, hi}, %4;\n\t"
      "cvt.rn.f16x2.e4m3x2 x, lo;\n\t"
      "cvt.rn.f16x2.e4m3x2 y, hi;\n\t"
      "mov.b32 {a, b}, x;\n\t"
      "mov.b32 {c, d}, y;\n\t"
      "cvt.f32.f16 %0, a;\n\t"
      "cvt.f32.f16 %1, b;\n\t"
      "cvt.f32.f16 %2, c;\n\t"
      "cvt.f32.f16 %3, d;\n\t}"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3])
      : "r"(q));
}
// One value to one code, one code to one value
__device__ __forceinline__ uint8_t pack1(float v) { return (uint8_t)pack4(v, 0.0f, 0.0f, 0.0f); }
__device__ __forceinline__ float unpack1(uint8_t q) {
  float v[4];
  unpack4(q, v);
  return v[0];
}

}  // namespace act8
}  // namespace moe
