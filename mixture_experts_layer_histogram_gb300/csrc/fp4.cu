// MXFP4 quantisation of a matrix, reading it back, and the token permutation that quantises on the
// way into the grouped layout. All three are HBM-bound passes over the data. A thread takes eight
// consecutive values (16 bytes of bf16), four lanes make one block of 32: the block's largest
// magnitude is two shuffles away, and the lanes' codes are consecutive 4-byte words. Sixteen lanes make
// one 128-value group, whose four scale bytes are one aligned word of the tiled scale layout.
#include "common.cuh"
#include "fp4.cuh"

namespace moe {
namespace fp4 {

constexpr int kThreads = 256;

// Eight consecutive values of a row as they lie in memory.
template <typename T> struct Raw8;
template <> struct Raw8<__nv_bfloat16> {
  uint4 q;
  __device__ __forceinline__ void zero() { q = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void load(const __nv_bfloat16 *p) { q = ld_stream(reinterpret_cast<const uint4 *>(p)); }
  __device__ __forceinline__ void unpack(float *v) const { unpack_bf16x8(q, v); }
  static __device__ __forceinline__ void store(__nv_bfloat16 *p, const float *v) {
    *reinterpret_cast<uint4 *>(p) = pack_bf16x8(v);
  }
};
template <> struct Raw8<float> {
  uint4 a, b;
  __device__ __forceinline__ void zero() { a = b = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void load(const float *p) {
    a = ld_stream(reinterpret_cast<const uint4 *>(p));
    b = ld_stream(reinterpret_cast<const uint4 *>(p) + 1);
  }
  __device__ __forceinline__ void unpack(float *v) const {
    v[0] = __uint_as_float(a.x); v[1] = __uint_as_float(a.y); v[2] = __uint_as_float(a.z); v[3] = __uint_as_float(a.w);
    v[4] = __uint_as_float(b.x); v[5] = __uint_as_float(b.y); v[6] = __uint_as_float(b.z); v[7] = __uint_as_float(b.w);
  }
  static __device__ __forceinline__ void store(float *p, const float *v) {
    reinterpret_cast<float4 *>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4 *>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
  }
};

// This lane's eight codes, and the four scale bytes of its group of sixteen lanes (the same in all of them).
template <typename T> __device__ __forceinline__ uint32_t quantize8(const Raw8<T> &raw, uint32_t &scales) {
  float v[8];
  raw.unpack(v);
  uint32_t amax = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) amax = max(amax, __float_as_uint(v[i]) & 0x7fffffffu);
  amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
  amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
  const uint32_t byte = scale_byte(amax);
  const float inv = inv_scale(byte);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = byte == 255u ? 0.0f : v[i] * inv;
  uint32_t s = byte << (8 * ((threadIdx.x >> 2) & 3));
  s |= __shfl_xor_sync(0xffffffffu, s, 4);
  s |= __shfl_xor_sync(0xffffffffu, s, 8);
  scales = s;
  return pack_e2m1x8(v);
}

// Block shape: `tpr` threads (a power of two, at least 16) per row, kThreads / tpr rows at a time.
struct Shape {
  int tpr_log2;
  int kgroups;     // groups of 128 values per row, the last one padded
};

// x [R, K] -> codes [R, K/2], scales (tiled). Rows from R up to the next multiple of 128 and values from K up
// to the next multiple of 128 have scale 0 and no codes.
template <typename T>
__global__ void __launch_bounds__(kThreads) quantize_kernel(const T *__restrict__ x, int64_t R, int64_t rows_pad, int K,
                                                            const Shape sh, uint8_t *__restrict__ codes,
                                                            uint8_t *__restrict__ scales) {
  const int tpr = 1 << sh.tpr_log2, rpb = kThreads >> sh.tpr_log2;
  const int lane_in_row = threadIdx.x & (tpr - 1), sub = threadIdx.x >> sh.tpr_log2;
  const int nvec = sh.kgroups * 16;
  for (int64_t r0 = (int64_t)blockIdx.x * rpb; r0 < rows_pad; r0 += (int64_t)gridDim.x * rpb) {
    const int64_t r = r0 + sub;     // rows_pad is a multiple of 128, so of rpb
    for (int v0 = 0; v0 < nvec; v0 += tpr) {
      const int v = v0 + lane_in_row;
      const bool in = r < R && v * 8 < K;
      Raw8<T> raw;
      raw.zero();
      if (in) raw.load(x + r * K + v * 8);
      uint32_t s;
      const uint32_t q = quantize8(raw, s);
      if (in) *reinterpret_cast<uint32_t *>(codes + r * (K / 2) + v * 4) = q;
      if (v < nvec && (v & 15) == 0) *reinterpret_cast<uint32_t *>(scales + scale_word(r, v >> 4, sh.kgroups)) = s;
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) dequantize_kernel(const uint8_t *__restrict__ codes,
                                                              const uint8_t *__restrict__ scales, int64_t R, int K,
                                                              const Shape sh, T *__restrict__ x) {
  const int tpr = 1 << sh.tpr_log2, rpb = kThreads >> sh.tpr_log2;
  const int lane_in_row = threadIdx.x & (tpr - 1), sub = threadIdx.x >> sh.tpr_log2;
  for (int64_t r = (int64_t)blockIdx.x * rpb + sub; r < R; r += (int64_t)gridDim.x * rpb) {
    for (int v = lane_in_row; v * 8 < K; v += tpr) {
      const uint32_t q = *reinterpret_cast<const uint32_t *>(codes + r * (K / 2) + v * 4);
      const float s = scale_value(scales[scale_word(r, v >> 4, sh.kgroups) + ((v >> 2) & 3)]);
      float f[8];
      unpack_e2m1x8(q, f);
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] *= s;
      Raw8<T>::store(x + r * K + v * 8, f);
    }
  }
}

// Tokens x [T, d] quantised once each and written to their k grouped rows; blocks past `token_blocks` write the
// padding rows of one expert (codes and scales zero).
template <typename T>
__global__ void __launch_bounds__(kThreads) permute_fp4_kernel(const T *__restrict__ x, int64_t Tn, int K,
                                                               const Shape sh, int k,
                                                               const int32_t *__restrict__ row_of_slot,
                                                               const int32_t *__restrict__ counts,
                                                               const int32_t *__restrict__ tile_offsets,
                                                               int64_t rows_max, int token_blocks,
                                                               uint8_t *__restrict__ codes,
                                                               uint8_t *__restrict__ scales) {
  const int tpr = 1 << sh.tpr_log2, rpb = kThreads >> sh.tpr_log2;
  const int lane_in_row = threadIdx.x & (tpr - 1), sub = threadIdx.x >> sh.tpr_log2;
  const int nvec = sh.kgroups * 16;
  if ((int)blockIdx.x >= token_blocks) {
    const int e = blockIdx.x - token_blocks;
    const int64_t start = (int64_t)tile_offsets[e] * kTileRows + counts[e];
    int64_t end = (int64_t)tile_offsets[e + 1] * kTileRows;
    if (end > rows_max) end = rows_max;
    for (int64_t r = start + sub; r < end; r += rpb) {
      for (int v = lane_in_row; v < nvec; v += tpr) {
        *reinterpret_cast<uint32_t *>(codes + r * (K / 2) + v * 4) = 0;
        if ((v & 15) == 0) *reinterpret_cast<uint32_t *>(scales + scale_word(r, v >> 4, sh.kgroups)) = 0;
      }
    }
    return;
  }
  for (int64_t t0 = (int64_t)blockIdx.x * rpb; t0 < Tn; t0 += (int64_t)token_blocks * rpb) {
    const int64_t t = t0 + sub;
    for (int v0 = 0; v0 < nvec; v0 += tpr) {
      const int v = v0 + lane_in_row;
      const bool in = t < Tn && v < nvec;
      Raw8<T> raw;
      raw.zero();
      if (in) raw.load(x + t * K + v * 8);
      uint32_t s;
      const uint32_t q = quantize8(raw, s);
      if (!in) continue;
      for (int j = 0; j < k; ++j) {
        const int64_t r = __ldg(row_of_slot + t * k + j);
        if (r < 0 || r >= rows_max) continue;
        *reinterpret_cast<uint32_t *>(codes + r * (K / 2) + v * 4) = q;
        if ((v & 15) == 0) *reinterpret_cast<uint32_t *>(scales + scale_word(r, v >> 4, sh.kgroups)) = s;
      }
    }
  }
}

static Shape shape_of(int K) {
  Shape s;
  s.kgroups = (K + 127) / 128;
  s.tpr_log2 = 4;
  while (s.tpr_log2 < 8 && (1 << s.tpr_log2) < s.kgroups * 16) ++s.tpr_log2;
  return s;
}

static int grid_for(int64_t rows, const Shape &s) {
  const int rpb = kThreads >> s.tpr_log2;
  int64_t b = (rows + rpb - 1) / rpb;
  const int64_t cap = (int64_t)sm_count() * 8;
  if (b > cap) b = cap;
  return b < 1 ? 1 : (int)b;
}

static int check(int64_t R, int K, int dtype) {
  if (R < 0 || K < 1 || (dtype != MOE_F32 && dtype != MOE_BF16)) return MOE_ERR_INVALID_ARG;
  if (K % kBlock) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}
static bool bad(const void *p) { return !p || !aligned16(p); }

}  // namespace fp4
}  // namespace moe

using namespace moe;
using namespace moe::fp4;

extern "C" size_t moe_fp4_scale_bytes(int64_t R, int K) {
  if (R < 0 || K < 1) return 0;
  return (size_t)((R + kTileRows - 1) / kTileRows) * (size_t)((K + 127) / 128) * kTileBytes;
}

extern "C" int moe_fp4_quantize(const void *x, int dtype, int64_t R, int K, void *codes, void *scales,
                                moe_stream_t stream) {
  const int rc = check(R, K, dtype);
  if (rc) return rc;
  if (R == 0) return MOE_OK;
  if (bad(x) || bad(codes) || bad(scales)) return MOE_ERR_INVALID_ARG;
  const Shape sh = shape_of(K);
  const int64_t rp = (R + kTileRows - 1) / kTileRows * kTileRows;
  cudaStream_t s = (cudaStream_t)stream;
  if (dtype == MOE_BF16)
    quantize_kernel<<<grid_for(rp, sh), kThreads, 0, s>>>((const __nv_bfloat16 *)x, R, rp, K, sh, (uint8_t *)codes,
                                                          (uint8_t *)scales);
  else
    quantize_kernel<<<grid_for(rp, sh), kThreads, 0, s>>>((const float *)x, R, rp, K, sh, (uint8_t *)codes,
                                                          (uint8_t *)scales);
  MOE_CHECK_LAUNCH();
  return MOE_OK;
}

extern "C" int moe_fp4_dequantize(const void *codes, const void *scales, int64_t R, int K, int dtype, void *x,
                                  moe_stream_t stream) {
  const int rc = check(R, K, dtype);
  if (rc) return rc;
  if (R == 0) return MOE_OK;
  if (bad(x) || bad(codes) || bad(scales)) return MOE_ERR_INVALID_ARG;
  const Shape sh = shape_of(K);
  cudaStream_t s = (cudaStream_t)stream;
  if (dtype == MOE_BF16)
    dequantize_kernel<<<grid_for(R, sh), kThreads, 0, s>>>((const uint8_t *)codes, (const uint8_t *)scales, R, K, sh,
                                                           (__nv_bfloat16 *)x);
  else
    dequantize_kernel<<<grid_for(R, sh), kThreads, 0, s>>>((const uint8_t *)codes, (const uint8_t *)scales, R, K, sh,
                                                           (float *)x);
  MOE_CHECK_LAUNCH();
  return MOE_OK;
}

extern "C" int moe_permute_fp4(const void *x, int dtype, int T, int d, int k, int E, const int32_t *row_of_slot,
                               const int32_t *counts, const int32_t *tile_offsets, int64_t rows_max, void *codes,
                               void *scales, moe_stream_t stream) {
  if (T < 0 || k < 1 || k > MOE_MAX_TOPK || E < 1 || E > MOE_MAX_EXPERTS) return MOE_ERR_INVALID_ARG;
  const int rc = check(T, d, dtype);
  if (rc) return rc;
  if (d % 128) return MOE_ERR_UNSUPPORTED;
  if (rows_max < moe_grouped_rows_max(T, k, E)) return MOE_ERR_INVALID_ARG;
  if (bad(codes) || bad(scales) || !counts || !tile_offsets || (T > 0 && (bad(x) || !row_of_slot)))
    return MOE_ERR_INVALID_ARG;
  const Shape sh = shape_of(d);
  const int tb = grid_for(T, sh);
  cudaStream_t s = (cudaStream_t)stream;
  if (dtype == MOE_BF16)
    permute_fp4_kernel<<<tb + E, kThreads, 0, s>>>((const __nv_bfloat16 *)x, (int64_t)T, d, sh, k, row_of_slot, counts,
                                                   tile_offsets, rows_max, tb, (uint8_t *)codes, (uint8_t *)scales);
  else
    permute_fp4_kernel<<<tb + E, kThreads, 0, s>>>((const float *)x, (int64_t)T, d, sh, k, row_of_slot, counts,
                                                   tile_offsets, rows_max, tb, (uint8_t *)codes, (uint8_t *)scales);
  MOE_CHECK_LAUNCH();
  return MOE_OK;
}
