// MXFP4 quantisation of a matrix, reading it back, and the token permutation that quantises on the
// way into the grouped layout: passes over the data, bound by HBM as long as the instructions per value
// stay few. A thread therefore takes sixteen consecutive values (half a block: one exchange with its
// neighbour gives the block's largest magnitude) and writes their codes as one 8-byte word; eight threads make
// one group of 128 values, whose four scale bytes are one aligned word of the tiled scale layout.
// Measured (bf16): quantising 16384 x 4096 takes 26.5 us (170 MB, 6.4 TB/s), permuting 8192 x 2048 to eight rows each
// 18.4 us (105 MB, 5.7 TB/s). With eight values per thread, two exchanges and 4-byte words they took 44.5 and 34.5 us.
#include "common.cuh"
#include "dependent.cuh"
#include "fp4.cuh"
#include "raw16.cuh"

namespace moe {
namespace fp4 {

constexpr int kThreads = 256;
constexpr int kVec = 16;          // values per thread
constexpr int kUnroll = 2;        // such vectors in flight per thread
constexpr int kPerBlock = kThreads * kUnroll;
constexpr int kGroupLanes = 128 / kVec;

// This lane's sixteen codes, and the four scale bytes of its group of eight lanes (the same in all of them).
template <typename T> __device__ __forceinline__ uint2 quantize16(const Raw16<T> &raw, uint32_t &scales) {
  uint32_t amax = raw.amax();
  amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
  const uint32_t byte = scale_byte(amax);
  const float inv = inv_scale(byte);
  uint32_t s = byte << (8 * ((threadIdx.x >> 1) & 3));
  s |= __shfl_xor_sync(0xffffffffu, s, 2);
  s |= __shfl_xor_sync(0xffffffffu, s, 4);
  scales = s;
  float v[16];
  raw.unpack(v);
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] *= inv;
  const uint2 q = make_uint2(pack_e2m1x8(v), pack_e2m1x8(v + 8));
  return byte == 255u ? make_uint2(0, 0) : q;
}

// Division by a fixed number d: for n < 2^31, n / d = (n * mul) >> shift with mul = floor(2^shift / d) + 1 and
// 2^(shift - 31) >= d.
struct Div {
  uint32_t d, shift;
  uint64_t mul;
  __device__ __forceinline__ uint32_t of(uint32_t n) const { return (uint32_t)((n * mul) >> shift); }
};
struct Shape {
  Div nvec;        // vectors of sixteen per row, padded to groups of 128 values
  int kgroups;
};

// x [R, K] -> codes [R, K/2], scales (tiled), for the `total` vectors from row row0 of the padded matrix on. Rows
// from R up to the next multiple of 128 and values from K up to the next multiple of 128 have scale 0 and no codes.
template <typename T>
__global__ void __launch_bounds__(kThreads) quantize_kernel(const T *__restrict__ x, int64_t R, int64_t row0,
                                                            uint32_t total, int K, const Shape sh,
                                                            uint8_t *__restrict__ codes, uint8_t *__restrict__ scales) {
  const uint32_t n0 = blockIdx.x * kPerBlock + threadIdx.x;
  Raw16<T> raw[kUnroll];
  int64_t r[kUnroll];
  int v[kUnroll];
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const uint32_t n = n0 + u * kThreads, q = sh.nvec.of(n);
    r[u] = row0 + q;
    v[u] = (int)(n - q * sh.nvec.d);
    raw[u].zero();
    if (n < total && r[u] < R && v[u] * kVec < K) raw[u].load(x + r[u] * K + v[u] * kVec);
  }
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    uint32_t s;
    const uint2 q = quantize16(raw[u], s);
    if (n0 + u * kThreads >= total) continue;
    if (r[u] < R && v[u] * kVec < K) *reinterpret_cast<uint2 *>(codes + r[u] * (K / 2) + v[u] * (kVec / 2)) = q;
    if (v[u] % kGroupLanes == 0)
      *reinterpret_cast<uint32_t *>(scales + scale_word(r[u], v[u] / kGroupLanes, sh.kgroups)) = s;
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) dequantize_kernel(const uint8_t *__restrict__ codes,
                                                              const uint8_t *__restrict__ scales, int64_t R,
                                                              int64_t row0, uint32_t total, int K, const Shape sh,
                                                              T *__restrict__ x) {
  const uint32_t n0 = blockIdx.x * kPerBlock + threadIdx.x;
  const bool wide = (reinterpret_cast<uintptr_t>(x) & 31) == 0;   // rows are multiples of 64 bytes
  uint2 q[kUnroll];
  uint32_t s[kUnroll];
  int64_t at[kUnroll];
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const uint32_t n = n0 + u * kThreads, rr = sh.nvec.of(n);
    const int64_t r = row0 + rr;
    const int v = (int)(n - rr * sh.nvec.d);
    at[u] = n < total && r < R && v * kVec < K ? r * K + v * kVec : -1;
    q[u] = make_uint2(0, 0);
    s[u] = 0;
    if (at[u] >= 0) {
      q[u] = __ldg(reinterpret_cast<const uint2 *>(codes + at[u] / 2));
      s[u] = __ldg(scales + scale_word(r, v / kGroupLanes, sh.kgroups) + ((v >> 1) & 3));
    }
  }
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    if (at[u] < 0) continue;
    const float sv = scale_value(s[u]);
    float f[16];
    unpack_e2m1x8(q[u].x, f);
    unpack_e2m1x8(q[u].y, f + 8);
#pragma unroll
    for (int i = 0; i < 16; ++i) f[i] *= sv;
    Raw16<T>::store(x + at[u], f, wide);
  }
}

// Tokens x [T, d] quantised once each and written to their k grouped rows, a warp per token and segment of 1024
// values: the token's rows are read once per warp, and its (up to) eight scale words of the segment are
// brought into lanes 0..7, which write them together. Blocks past `token_blocks` write the padding rows (codes and
// scales zero), 32 rows of one expert each.
constexpr int kPadRows = 32;
constexpr int kSegVecs = 32 * kUnroll;
template <typename T>
__global__ void __launch_bounds__(kThreads) permute_fp4_kernel(const T *__restrict__ x, uint32_t units, int K,
                                                               const Div nseg, int nvec, int k,
                                                               const int32_t *__restrict__ row_of_slot,
                                                               const int32_t *__restrict__ counts,
                                                               const int32_t *__restrict__ tile_offsets,
                                                               int64_t rows_max, int token_blocks,
                                                               uint8_t *__restrict__ codes,
                                                               uint8_t *__restrict__ scales) {
  start_next();   // the grouped FFN may set up and fetch weights meanwhile
  const int kgroups = K / 128;
  if ((int)blockIdx.x >= token_blocks) {
    const int b = blockIdx.x - token_blocks, e = b / (kTileRows / kPadRows), part = b % (kTileRows / kPadRows);
    const int64_t start = (int64_t)tile_offsets[e] * kTileRows + counts[e] + part * kPadRows;
    int64_t end = (int64_t)tile_offsets[e + 1] * kTileRows;
    if (end > rows_max) end = rows_max;
    if (end > start + kPadRows) end = start + kPadRows;
    if (start < 0 || start >= end) return;
    uint4 *dst = reinterpret_cast<uint4 *>(codes + start * (K / 2));
    for (int64_t i = threadIdx.x; i < (end - start) * (K / 32); i += kThreads) dst[i] = make_uint4(0, 0, 0, 0);
    for (int i = threadIdx.x; i < (int)(end - start) * kgroups; i += kThreads) {
      const int rr = i / kgroups;
      *reinterpret_cast<uint32_t *>(scales + scale_word(start + rr, i - rr * kgroups, kgroups)) = 0;
    }
    return;
  }
  const int lane = threadIdx.x & 31;
  const uint32_t unit = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  if (unit >= units) return;
  const uint32_t t = nseg.of(unit);
  const int v0 = (int)(unit - t * nseg.d) * kSegVecs;      // first vector of the segment
  int myrow = -1;
  if (lane < k) {
    myrow = __ldg(row_of_slot + (int64_t)t * k + lane);
    if (myrow >= rows_max) myrow = -1;
  }
  Raw16<T> raw[kUnroll];
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const int v = v0 + u * 32 + lane;
    raw[u].zero();
    if (v < nvec) raw[u].load(x + (int64_t)t * K + v * kVec);
  }
  uint2 q[kUnroll];
  uint32_t word = 0;                                       // lane l < 8: scales of group l of the segment
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    uint32_t s;
    q[u] = quantize16(raw[u], s);
    const uint32_t w = __shfl_sync(0xffffffffu, s, (lane & 3) * kGroupLanes);
    if ((lane >> 2) == u) word = w;
  }
  const int group = v0 / kGroupLanes + lane;
  for (int j = 0; j < k; ++j) {
    const int r = __shfl_sync(0xffffffffu, myrow, j);
    if (r < 0) continue;
    uint8_t *dst = codes + (int64_t)r * (K / 2) + (v0 + lane) * (kVec / 2);
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
      if (v0 + u * 32 + lane < nvec) *reinterpret_cast<uint2 *>(dst + u * 32 * (kVec / 2)) = q[u];
    if (lane < 4 * kUnroll && group < kgroups)
      *reinterpret_cast<uint32_t *>(scales + scale_word(r, group, kgroups)) = word;
  }
}

static Div div_by(int d) {
  Div v;
  v.d = (uint32_t)d;
  int l = 0;
  while ((1 << l) < d) ++l;
  v.shift = 31 + l;
  v.mul = ((uint64_t)1 << v.shift) / (uint64_t)d + 1;
  return v;
}

static Shape shape_of(int K) {
  Shape s;
  s.kgroups = (K + 127) / 128;
  s.nvec = div_by(s.kgroups * kGroupLanes);
  return s;
}

// Rows per launch: vectors are numbered in 31 bits.
static int64_t rows_per_launch(const Shape &s) { return (((int64_t)1 << 31) - kPerBlock) / s.nvec.d / kTileRows * kTileRows; }
static int blocks_for(uint32_t total) { return (int)((total + kPerBlock - 1) / kPerBlock); }

static int check(int64_t R, int K, int dtype) {
  if (R < 0 || K < 1 || (dtype != MOE_F32 && dtype != MOE_BF16)) return MOE_ERR_INVALID_ARG;
  if (K % kBlock || K > (1 << 26)) return MOE_ERR_UNSUPPORTED;   // rows_per_launch is at least 128 below that
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
  const int64_t rp = (R + kTileRows - 1) / kTileRows * kTileRows, most = rows_per_launch(sh);
  cudaStream_t s = (cudaStream_t)stream;
  for (int64_t r0 = 0; r0 < rp; r0 += most) {
    const uint32_t total = (uint32_t)((rp - r0 < most ? rp - r0 : most) * sh.nvec.d);
    if (dtype == MOE_BF16)
      quantize_kernel<<<blocks_for(total), kThreads, 0, s>>>((const __nv_bfloat16 *)x, R, r0, total, K, sh,
                                                             (uint8_t *)codes, (uint8_t *)scales);
    else
      quantize_kernel<<<blocks_for(total), kThreads, 0, s>>>((const float *)x, R, r0, total, K, sh, (uint8_t *)codes,
                                                             (uint8_t *)scales);
    MOE_CHECK_LAUNCH();
  }
  return MOE_OK;
}

extern "C" int moe_fp4_dequantize(const void *codes, const void *scales, int64_t R, int K, int dtype, void *x,
                                  moe_stream_t stream) {
  const int rc = check(R, K, dtype);
  if (rc) return rc;
  if (R == 0) return MOE_OK;
  if (bad(x) || bad(codes) || bad(scales)) return MOE_ERR_INVALID_ARG;
  const Shape sh = shape_of(K);
  const int64_t most = rows_per_launch(sh);
  cudaStream_t s = (cudaStream_t)stream;
  for (int64_t r0 = 0; r0 < R; r0 += most) {
    const uint32_t total = (uint32_t)((R - r0 < most ? R - r0 : most) * sh.nvec.d);
    if (dtype == MOE_BF16)
      dequantize_kernel<<<blocks_for(total), kThreads, 0, s>>>((const uint8_t *)codes, (const uint8_t *)scales, R, r0,
                                                               total, K, sh, (__nv_bfloat16 *)x);
    else
      dequantize_kernel<<<blocks_for(total), kThreads, 0, s>>>((const uint8_t *)codes, (const uint8_t *)scales, R, r0,
                                                               total, K, sh, (float *)x);
    MOE_CHECK_LAUNCH();
  }
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
  const int nvec = d / kVec, segs = (nvec + kSegVecs - 1) / kSegVecs;
  if ((int64_t)T * segs >= ((int64_t)1 << 31) - kThreads) return MOE_ERR_UNSUPPORTED;
  const uint32_t units = (uint32_t)T * (uint32_t)segs;
  const int tb = (int)((units + kThreads / 32 - 1) / (kThreads / 32)), grid = tb + E * (kTileRows / kPadRows);
  const Div by = div_by(segs);
  cudaStream_t s = (cudaStream_t)stream;
  if (dtype == MOE_BF16)
    permute_fp4_kernel<<<grid, kThreads, 0, s>>>((const __nv_bfloat16 *)x, units, d, by, nvec, k, row_of_slot, counts,
                                                 tile_offsets, rows_max, tb, (uint8_t *)codes, (uint8_t *)scales);
  else
    permute_fp4_kernel<<<grid, kThreads, 0, s>>>((const float *)x, units, d, by, nvec, k, row_of_slot, counts,
                                                 tile_offsets, rows_max, tb, (uint8_t *)codes, (uint8_t *)scales);
  MOE_CHECK_LAUNCH();
  return MOE_OK;
}
