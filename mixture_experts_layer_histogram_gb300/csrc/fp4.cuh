// MXFP4 in registers: blocks of 32 values along K, one E8M0 scale per block (byte b stands for
// 2^(b - 127), 0xff for NaN), E2M1 codes (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives).
//
// The scale of a block is 2^(floor(log2 max|x|) - 2) (OCP Microscaling Formats, version 1.0: the
// largest E2M1 exponent is 2), so max|x| / scale lies in [4, 8); what exceeds 6 saturates. In bits:
// the exponent field of max|x| less two, not below zero. Dividing by a power of two is exact, so codes
// depend on the input alone.
#pragma once

#include "common.cuh"

namespace moe {
namespace fp4 {

constexpr int kBlock = 32;        // values per scale
constexpr int kTileRows = 128;    // rows, and ...
constexpr int kTileBlocks = 4;    // ... blocks along K, per 512-byte tile of scales
constexpr int kTileBytes = kTileRows * kTileBlocks;

// Byte of row r (of its 128-row tile) and block kb (of its group of four) inside a 512-byte scale tile:
// the order in which the tensor cores take a 128-row operand's scales from shared memory.
__host__ __device__ __forceinline__ int scale_in_tile(int r, int kb) { return (r & 31) * 16 + (r >> 5) * 4 + kb; }

// Offset of the four scales of row r, K group kg (of kgroups groups of 128 values); four bytes, one per block.
__device__ __forceinline__ int64_t scale_word(int64_t r, int kg, int kgroups) {
  return ((r >> 7) * kgroups + kg) * kTileBytes + scale_in_tile((int)(r & 127), 0);
}

// Scale byte of a block whose largest magnitude has the fp32 bits `amax` (sign clear). NaN bits are the
// largest integers, so an integer maximum carries a NaN through, and a non-finite block gets 0xff.
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax) {
  const int e = (int)(amax >> 23);
  return e == 255 ? 255u : (uint32_t)(e > 2 ? e - 2 : 0);
}
// 1 / scale as fp32 (0 for a NaN block: its codes are zeros)
__device__ __forceinline__ float inv_scale(uint32_t byte) { return __uint_as_float(byte == 255u ? 0u : (254u - byte) << 23); }
// The scale as fp32
__device__ __forceinline__ float scale_value(uint32_t byte) {
  return __uint_as_float(byte == 255u ? 0x7fc00000u : (byte == 0 ? 0x00400000u : byte << 23));
}

// Eight values to eight E2M1 codes (round to nearest even, saturating), the first in the low bits.
__device__ __forceinline__ uint32_t pack_e2m1x8(const float *v) {
  uint32_t r;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}
// Eight codes to eight values
__device__ __forceinline__ void unpack_e2m1x8(uint32_t q, float *v) {
  uint32_t h[4];
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(q));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    asm("{\n\t.reg .b16 lo, hi;\n\t"
        "mov.b32 {lo, hi}, %2;\n\t"
        "cvt.f32.f16 %0, lo;\n\t"
        "cvt.f32.f16 %1, hi;\n\t}"
        : "=f"(v[2 * i]), "=f"(v[2 * i + 1])
        : "r"(h[i]));
  }
}

}  // namespace fp4
}  // namespace moe
