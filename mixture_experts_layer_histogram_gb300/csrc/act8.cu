// Activations to 8 bits and back: passes over the data, bound by HBM while the instructions per value stay few.
//
// Rows of whole blocks (K a multiple of 32) are one flat array: a thread takes sixteen consecutive values, half a block,
// and one exchange with its neighbour gives the block's largest magnitude; codes leave as one 16-byte word. Other
// row lengths take a warp per block of 32 with one value per lane.
// Measured at 16384 x 4096 bf16 (203 MB each way, HBM at 93% of the copy rate): 28 us to 8 bits, 28 back, 65.5 together; 77 x
// 999 fp32 4.3 and 4.8 us, in a stream of calls 11.3 together (the host's two calls). Large rows that are no multiple of 32 are bound by
// instructions (a load, a store and a share of a division per value): 16384 x 4099 364 us there and back, bf16 or fp32, where the bytes
// take 61 or 101.
#include "act8.cuh"
#include "common.cuh"
#include "raw16.cuh"

namespace moe {
namespace act8 {

constexpr int kThreads = 256;
constexpr int kVec = 16;          // values per thread
constexpr int kUnroll = 2;        // such vectors in flight per thread
constexpr int kPerBlock = kThreads * kUnroll;

// n half blocks of a flat array
template <typename T>
__global__ void __launch_bounds__(kThreads) quantize_kernel(const T *__restrict__ x, int64_t n, uint4 *__restrict__ codes,
                                                            uint8_t *__restrict__ scales) {
  const int64_t n0 = (int64_t)blockIdx.x * kPerBlock + threadIdx.x;
  Raw16<T> raw[kUnroll];
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    raw[u].zero();
    if (n0 + u * kThreads < n) raw[u].load(x + (n0 + u * kThreads) * kVec);
  }
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const int64_t at = n0 + u * kThreads;
    uint32_t amax = raw[u].amax();
    amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    const uint32_t byte = scale_byte(amax);
    const float inv = inv_scale(byte);
    float v[16];
    raw[u].unpack(v);
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] *= inv;
    uint4 q = make_uint4(pack4(v[0], v[1], v[2], v[3]), pack4(v[4], v[5], v[6], v[7]), pack4(v[8], v[9], v[10], v[11]),
                         pack4(v[12], v[13], v[14], v[15]));
    if (byte == 255u) q = make_uint4(0, 0, 0, 0);
    if (at >= n) continue;
    codes[at] = q;
    if ((at & 1) == 0) scales[at >> 1] = (uint8_t)byte;
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) dequantize_kernel(const uint4 *__restrict__ codes,
                                                              const uint8_t *__restrict__ scales, int64_t n,
                                                              T *__restrict__ x) {
  const int64_t n0 = (int64_t)blockIdx.x * kPerBlock + threadIdx.x;
  const bool wide = (reinterpret_cast<uintptr_t>(x) & 31) == 0;
  uint4 q[kUnroll];
  uint32_t s[kUnroll];
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const int64_t at = n0 + u * kThreads;
    q[u] = make_uint4(0, 0, 0, 0);
    s[u] = 0;
    if (at < n) {
      q[u] = __ldg(codes + at);
      s[u] = __ldg(scales + (at >> 1));
    }
  }
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const int64_t at = n0 + u * kThreads;
    if (at >= n) continue;
    const float sv = scale_value(s[u]);
    float v[16];
    unpack4(q[u].x, v);
    unpack4(q[u].y, v + 4);
    unpack4(q[u].z, v + 8);
    unpack4(q[u].w, v + 12);
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] *= sv;
    Raw16<T>::store(x + at * kVec, v, wide);
  }
}

__device__ __forceinline__ void put(float *p, float v) { *p = v; }
__device__ __forceinline__ void put(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }

// Any row length: a warp per block, warps numbered through all rows' blocks.
template <typename T>
__global__ void __launch_bounds__(kThreads) quantize_any_kernel(const T *__restrict__ x, int64_t total, int K, int nb,
                                                                uint8_t *__restrict__ codes, uint8_t *__restrict__ scales) {
  const int lane = threadIdx.x & 31;
  const int64_t step = (int64_t)gridDim.x * (kThreads / 32);
  for (int64_t b = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); b < total; b += step) {
    const int64_t r = b / nb;
    const int c = (int)(b - r * nb) * kBlock + lane;
    const float v = c < K ? (float)x[r * K + c] : 0.0f;
    const uint32_t byte = scale_byte(__reduce_max_sync(0xffffffffu, __float_as_uint(v) & 0x7fffffffu));
    if (c < K) codes[r * K + c] = byte == 255u ? (uint8_t)0 : pack1(v * inv_scale(byte));
    if (lane == 0) scales[b] = (uint8_t)byte;
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) dequantize_any_kernel(const uint8_t *__restrict__ codes,
                                                                  const uint8_t *__restrict__ scales, int64_t total, int K,
                                                                  int nb, T *__restrict__ x) {
  const int lane = threadIdx.x & 31;
  const int64_t step = (int64_t)gridDim.x * (kThreads / 32);
  for (int64_t b = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); b < total; b += step) {
    const int64_t r = b / nb;
    const int c = (int)(b - r * nb) * kBlock + lane;
    if (c < K) put(x + r * K + c, unpack1(codes[r * K + c]) * scale_value(scales[b]));
  }
}

static int check(int64_t R, int K, int dtype) {
  if (R < 0 || K < 1 || (dtype != MOE_F32 && dtype != MOE_BF16)) return MOE_ERR_INVALID_ARG;
  if (R > ((int64_t)1 << 39) / K) return MOE_ERR_UNSUPPORTED;   // the flat kernels' block number has 31 bits
  return MOE_OK;
}
static bool bad(const void *p) { return !p || !aligned16(p); }
static unsigned any_grid(int64_t total) {
  const int64_t want = (total + kThreads / 32 - 1) / (kThreads / 32), most = (int64_t)sm_count() * 8;
  return (unsigned)(want < most ? want : most);
}

template <typename T>
static void quantize(const void *x, int64_t R, int K, void *codes, void *scales, cudaStream_t s) {
  if (K % kBlock == 0) {
    const int64_t n = R * (K / kVec);
    quantize_kernel<<<(unsigned)((n + kPerBlock - 1) / kPerBlock), kThreads, 0, s>>>((const T *)x, n, (uint4 *)codes,
                                                                                  (uint8_t *)scales);
  } else {
    const int nb = (int)blocks_of(K);
    quantize_any_kernel<<<any_grid(R * nb), kThreads, 0, s>>>((const T *)x, R * nb, K, nb, (uint8_t *)codes,
                                                              (uint8_t *)scales);
  }
}
template <typename T>
static void dequantize(const void *codes, const void *scales, int64_t R, int K, void *x, cudaStream_t s) {
  if (K % kBlock == 0) {
    const int64_t n = R * (K / kVec);
    dequantize_kernel<<<(unsigned)((n + kPerBlock - 1) / kPerBlock), kThreads, 0, s>>>((const uint4 *)codes,
                                                                                    (const uint8_t *)scales, n, (T *)x);
  } else {
    const int nb = (int)blocks_of(K);
    dequantize_any_kernel<<<any_grid(R * nb), kThreads, 0, s>>>((const uint8_t *)codes, (const uint8_t *)scales, R * nb,
                                                                K, nb, (T *)x);
  }
}

}  // namespace act8
}  // namespace moe

using namespace moe;
using namespace moe::act8;

extern "C" size_t moe_act8_scale_bytes(int64_t R, int K) {
  if (R < 0 || K < 1) return 0;
  return (size_t)R * (size_t)blocks_of(K);
}

extern "C" int moe_act8_quantize(const void *x, int dtype, int64_t R, int K, void *codes, void *scales,
                                 moe_stream_t stream) {
  const int rc = check(R, K, dtype);
  if (rc) return rc;
  if (R == 0) return MOE_OK;
  if (bad(x) || bad(codes) || bad(scales)) return MOE_ERR_INVALID_ARG;
  if (dtype == MOE_BF16) quantize<__nv_bfloat16>(x, R, K, codes, scales, (cudaStream_t)stream);
  else quantize<float>(x, R, K, codes, scales, (cudaStream_t)stream);
  MOE_CHECK_LAUNCH();
  return MOE_OK;
}

extern "C" int moe_act8_dequantize(const void *codes, const void *scales, int64_t R, int K, int dtype, void *x,
                                   moe_stream_t stream) {
  const int rc = check(R, K, dtype);
  if (rc) return rc;
  if (R == 0) return MOE_OK;
  if (bad(x) || bad(codes) || bad(scales)) return MOE_ERR_INVALID_ARG;
  if (dtype == MOE_BF16) dequantize<__nv_bfloat16>(codes, scales, R, K, x, (cudaStream_t)stream);
  else dequantize<float>(codes, scales, R, K, x, (cudaStream_t)stream);
  MOE_CHECK_LAUNCH();
  return MOE_OK;
}
