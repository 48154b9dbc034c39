// One AdamW step over many tensors in one launch per kind of tensor, states in fp32 or in 8 bits.
//
//   m' = b1 m + (1 - b1) c g,   v' = b2 v + (1 - b2) (c g)^2,   c = grad_scale
//   p' = p (1 - lr wd) - lr (m' / (1 - b1^t)) / (sqrt(v' / (1 - b2^t)) + eps)
//
// HBM-bound: every value is read and written once. The tensors are cut into chunks of 4096 values; a
// plan made on the host lists them, so a launch covers any number of tensors of any size and a block
// finds its tensor with two dependent loads. The bias corrections come from the step count in device
// memory, which the launch's last block advances: a captured step counts on when it is replayed.
//
// 8-bit states: blocks of 256 consecutive values share one fp32 scale, max / 448; m is held as e4m3
// codes of m / scale, v as e4m3 codes of sqrt(v) / scale (the root halves the range of exponents: e4m3
// spans 2^18, so v spans 2^36 within a block). A warp owns one block of 256. m, v and the update are computed in fp32
// from the decoded values and the parameter uses the new m and v before they are rounded.
//
// Dithered rounding. Rounding to nearest would hold v still: with b2 = 0.999 a step moves sqrt(v) by
// about 0.05%, and half an e4m3 step is 3-6%. Values kept in few bits only (e4m3 states, bf16
// parameters without an fp32 master copy) are rounded down after adding u of a step, u from the Weyl
// sequence (i A + t B) mod 2^32 over the place in the tensor and the step count: over the steps u is
// spread evenly, so the rounded value is right on average. The three uses take the sequence a third
// of its period apart.
#include <cuda_fp8.h>

#include <cmath>
#include <type_traits>

#include "common.cuh"

namespace moe {
namespace adamw {

constexpr int kThreads = 256;
constexpr int kChunk = 4096;      // values per chunk: two passes of 8 values per thread
constexpr int kVec = 8;
constexpr int kBlockQ = MOE_ADAMW_BLOCK;
static_assert(kBlockQ == 32 * kVec, "a warp owns one block of an 8-bit state");

// Kinds of tensors: parameter and gradient type, fp32 master copy, state.
enum Kind { F32_F32 = 0, BF16_F32, BF16_MASTER_F32, F32_F8, BF16_F8, BF16_MASTER_F8, KINDS };

struct Chunk {
  int32_t tensor, index;          // values [index * kChunk, ...) of the tensor
};
struct Tensor {                   // device form of moe_adamw_tensor
  void *p;
  float *master;
  const void *g;
  void *m, *v;
  float *m_scale, *v_scale;
  int64_t n;
  float weight_decay;
  int32_t aligned;                // every pointer allows vector access
};
struct Header {                   // at the start of a plan; the tensors and then the chunks follow
  int32_t magic, count;
  int64_t chunks[KINDS];
  int64_t chunks_at;              // byte offset of the chunk list (kind after kind)
};
constexpr int32_t kMagic = 0x41644d57;

struct Hyper {
  float beta1, beta2, omb1, omb2, eps, log_beta1, log_beta2;   // omb: 1 - beta, from the host's doubles
};

__device__ __forceinline__ uint32_t weyl(uint32_t i, uint32_t t) { return i * 2654435769u + t * 1640531535u; }

// y (|y| <= 448) to e4m3 codes, rounded down on the grid of its binade after adding u20 / 2^20 of a step.
__device__ __forceinline__ float dither_e4m3(float y, uint32_t u20) {
  const float a = fabsf(y);
  const float normal = __uint_as_float((__float_as_uint(a) + u20) & 0xfff00000u);
  const float small = (float)((__float2int_rz(a * 536870912.0f) + (int)u20) >> 20) * 0.001953125f;   // steps of 2^-9
  const float r = a < 0.015625f ? small : normal;
  return y != y ? y : copysignf(fminf(r, 448.0f), y);
}
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {   // exact here: the values lie on the grid
  return (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ void unpack_e4m3x8(const uint2 &q, float *v) {
  const uint32_t w[2] = {q.x, q.y};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w[i >> 1] >> (16 * (i & 1))), __NV_E4M3);
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}
// A bf16 value as the upper half of an fp32 word, rounded down in magnitude after adding u16 / 2^16 of a step.
__device__ __forceinline__ uint32_t dither_bf16_bits(float p, uint32_t u16) {
  const uint32_t b = __float_as_uint(p);
  if ((b & 0x7f800000u) == 0x7f800000u) return p != p ? 0x7fff0000u : b;   // NaN, infinity
  return (b + u16) & 0xffff0000u;
}

__device__ __forceinline__ void load8(const float *p, float *v) {
  const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w; v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ void store8(float *p, const float *v) {
  reinterpret_cast<float4 *>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4 *>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void load8(const __nv_bfloat16 *p, float *v) {
  unpack_bf16x8(*reinterpret_cast<const uint4 *>(p), v);
}
template <typename T> __device__ __forceinline__ float load1(const T *p) {
  if constexpr (sizeof(T) == 4) return *p;
  else return __bfloat162float(*p);
}

template <int K>
__global__ void __launch_bounds__(kThreads) adamw_kernel(const Tensor *__restrict__ tensors,
                                                         const Chunk *__restrict__ chunks, int64_t nchunks,
                                                         const Hyper hy, moe_adamw_state *st, int bump) {
  constexpr bool kF8 = K >= F32_F8;
  constexpr bool kMaster = K == BF16_MASTER_F32 || K == BF16_MASTER_F8;
  constexpr bool kF32 = K == F32_F32 || K == F32_F8;
  using T = typename std::conditional<kF32, float, __nv_bfloat16>::type;
  const int lane = threadIdx.x & 31;
  const int64_t step = st->step + 1;
  const float lr = st->lr, gs = st->grad_scale;
  const float bc1 = -expm1f((float)step * hy.log_beta1), bc2 = -expm1f((float)step * hy.log_beta2);
  const float lr1 = lr / bc1, inv_root2 = 1.0f / sqrtf(bc2);
  const uint32_t t32 = (uint32_t)step;

  for (int64_t ci = blockIdx.x; ci < nchunks; ci += gridDim.x) {
    const Chunk ch = chunks[ci];
    const Tensor t = tensors[ch.tensor];
    const float decay = 1.0f - lr * t.weight_decay;
    const T *gp = (const T *)t.g;
    T *pp = (T *)t.p;
#pragma unroll
    for (int pass = 0; pass < kChunk / (kThreads * kVec); ++pass) {
      const int64_t i0 = (int64_t)ch.index * kChunk + pass * (kThreads * kVec) + threadIdx.x * kVec;
      if (i0 - lane * kVec >= t.n) continue;              // the whole warp lies past the end
      const int64_t left = t.n - i0;
      const int live = left >= kVec ? kVec : (left > 0 ? (int)left : 0);
      const bool vec = live == kVec && t.aligned;
      float g[kVec], p[kVec], m[kVec], v[kVec];
      float ms = 0.0f, vs = 0.0f;
      const int64_t qb = i0 / kBlockQ;
      if (kF8) {
        ms = t.m_scale[qb];
        vs = t.v_scale[qb];
      }
      if (vec) {
        load8(gp + i0, g);
        if (kMaster) load8(t.master + i0, p);
        else load8(pp + i0, p);
        if (kF8) {
          unpack_e4m3x8(*reinterpret_cast<const uint2 *>((const uint8_t *)t.m + i0), m);
          unpack_e4m3x8(*reinterpret_cast<const uint2 *>((const uint8_t *)t.v + i0), v);
        } else {
          load8((const float *)t.m + i0, m);
          load8((const float *)t.v + i0, v);
        }
      } else {
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
          g[j] = p[j] = m[j] = v[j] = 0.0f;
          if (j >= live) continue;
          g[j] = load1(gp + i0 + j);
          p[j] = kMaster ? t.master[i0 + j] : load1(pp + i0 + j);
          if (kF8) {
            m[j] = (float)((const __nv_fp8_e4m3 *)t.m)[i0 + j];
            v[j] = (float)((const __nv_fp8_e4m3 *)t.v)[i0 + j];
          } else {
            m[j] = ((const float *)t.m)[i0 + j];
            v[j] = ((const float *)t.v)[i0 + j];
          }
        }
      }
      float mx = 0.0f, vx = 0.0f;
#pragma unroll
      for (int j = 0; j < kVec; ++j) {
        const float gj = g[j] * gs;
        if (kF8) {
          m[j] *= ms;
          v[j] *= vs;
          v[j] *= v[j];
        }
        m[j] = hy.beta1 * m[j] + hy.omb1 * gj;
        v[j] = hy.beta2 * v[j] + hy.omb2 * (gj * gj);
        const float root = sqrtf(v[j]);
        p[j] = p[j] * decay - lr1 * m[j] / (root * inv_root2 + hy.eps);
        if (kF8) {
          v[j] = root;
          mx = fmaxf(mx, fabsf(m[j]));
          vx = fmaxf(vx, root);
        }
      }
      float mi = 0.0f, vi = 0.0f;
      if (kF8) {
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) {
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
          vx = fmaxf(vx, __shfl_xor_sync(0xffffffffu, vx, off));
        }
        mi = mx >= 1e-30f ? 448.0f / mx : 0.0f;   // below it the block is held as zeros
        vi = vx >= 1e-30f ? 448.0f / vx : 0.0f;
        if (lane == 0) {
          t.m_scale[qb] = mx >= 1e-30f ? mx / 448.0f : 0.0f;
          t.v_scale[qb] = vx >= 1e-30f ? vx / 448.0f : 0.0f;
        }
      }
      uint32_t pb[kVec];
#pragma unroll
      for (int j = 0; j < kVec; ++j) {
        const uint32_t h = weyl((uint32_t)i0 + j, t32);
        if (kF8) {
          m[j] = dither_e4m3(m[j] * mi, h >> 12);
          v[j] = dither_e4m3(v[j] * vi, (h + 0x55555555u) >> 12);
        }
        if (!kF32 && !kMaster) pb[j] = dither_bf16_bits(p[j], (h + 0xaaaaaaaau) >> 16);
        if (kMaster) pb[j] = (uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(p[j])) << 16;
      }
      if (vec) {
        if constexpr (kF32) {
          store8((float *)t.p + i0, p);
        } else {
          *reinterpret_cast<uint4 *>(pp + i0) =
              make_uint4((pb[0] >> 16) | pb[1], (pb[2] >> 16) | pb[3], (pb[4] >> 16) | pb[5], (pb[6] >> 16) | pb[7]);
          if (kMaster) store8(t.master + i0, p);
        }
        if (kF8) {
          *reinterpret_cast<uint2 *>((uint8_t *)t.m + i0) =
              make_uint2(e4m3x2(m[0], m[1]) | e4m3x2(m[2], m[3]) << 16, e4m3x2(m[4], m[5]) | e4m3x2(m[6], m[7]) << 16);
          *reinterpret_cast<uint2 *>((uint8_t *)t.v + i0) =
              make_uint2(e4m3x2(v[0], v[1]) | e4m3x2(v[2], v[3]) << 16, e4m3x2(v[4], v[5]) | e4m3x2(v[6], v[7]) << 16);
        } else {
          store8((float *)t.m + i0, m);
          store8((float *)t.v + i0, v);
        }
      } else {
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
          if (j >= live) continue;
          if constexpr (kF32) {
            ((float *)t.p)[i0 + j] = p[j];
          } else {
            pp[i0 + j] = __ushort_as_bfloat16((unsigned short)(pb[j] >> 16));
            if (kMaster) t.master[i0 + j] = p[j];
          }
          if (kF8) {
            ((uint8_t *)t.m)[i0 + j] = (uint8_t)e4m3x2(m[j], 0.0f);
            ((uint8_t *)t.v)[i0 + j] = (uint8_t)e4m3x2(v[j], 0.0f);
          } else {
            ((float *)t.m)[i0 + j] = m[j];
            ((float *)t.v)[i0 + j] = v[j];
          }
        }
      }
    }
  }
  // every thread of a block has read the step count when the block arrives; the last block advances it
  __syncthreads();
  if (bump && threadIdx.x == 0) {
    __threadfence();
    if (atomicAdd(&st->arrived, 1u) == gridDim.x - 1) {
      st->arrived = 0;
      st->step = step;
    }
  }
}

static int kind_of(const moe_adamw_tensor &t) {
  const int base = t.dtype == MOE_F32 ? 0 : (t.master ? 2 : 1);
  return base + (t.state == MOE_ADAMW_F8 ? 3 : 0);
}

static int check(const moe_adamw_tensor &t) {
  if (t.n < 0 || (t.dtype != MOE_F32 && t.dtype != MOE_BF16) || (t.state != MOE_ADAMW_F32 && t.state != MOE_ADAMW_F8))
    return MOE_ERR_INVALID_ARG;
  if (!(t.weight_decay >= 0.0f)) return MOE_ERR_INVALID_ARG;
  if (t.dtype == MOE_F32 && t.master) return MOE_ERR_INVALID_ARG;
  if (t.n == 0) return MOE_OK;
  const uintptr_t es = t.dtype == MOE_F32 ? 4 : 2, ss = t.state == MOE_ADAMW_F32 ? 4 : 1;
  auto is = [](const void *p, uintptr_t a) { return p && (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; };
  if (!is(t.p, es) || !is(t.g, es) || !is(t.m, ss) || !is(t.v, ss) || (t.master && !is(t.master, 4)))
    return MOE_ERR_INVALID_ARG;
  if (t.state == MOE_ADAMW_F8 && (!is(t.m_scale, 4) || !is(t.v_scale, 4))) return MOE_ERR_INVALID_ARG;
  if ((t.n + kChunk - 1) / kChunk >= ((int64_t)1 << 31)) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

template <int K>
static int launch(const uint8_t *dev, const Header *h, int64_t first, int64_t n, const Hyper &hy, moe_adamw_state *st,
                  bool bump, cudaStream_t s) {
  int per_sm = 0;
  MOE_TRY_CUDA(cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, adamw_kernel<K>, kThreads, 0));
  int64_t grid = (int64_t)sm_count() * per_sm;
  if (grid > n) grid = n;
  if (grid < 1) grid = 1;
  adamw_kernel<K><<<(int)grid, kThreads, 0, s>>>((const Tensor *)(dev + sizeof(Header)),
                                                 (const Chunk *)(dev + h->chunks_at) + first, n, hy, st, bump ? 1 : 0);
  MOE_CHECK_LAUNCH();
  return MOE_OK;
}

}  // namespace adamw
}  // namespace moe

using namespace moe;
using namespace moe::adamw;

extern "C" size_t moe_adamw_plan_size(const moe_adamw_tensor *tensors, int count) {
  if (count < 0 || (count > 0 && !tensors)) return 0;
  size_t chunks = 0;
  for (int i = 0; i < count; ++i)
    if (tensors[i].n > 0) chunks += (size_t)((tensors[i].n + kChunk - 1) / kChunk);
  return sizeof(Header) + (size_t)count * sizeof(Tensor) + chunks * sizeof(Chunk);
}

extern "C" int moe_adamw_plan(const moe_adamw_tensor *tensors, int count, void *plan, size_t plan_bytes) {
  if (count < 0 || (count > 0 && !tensors) || !plan || (reinterpret_cast<uintptr_t>(plan) & 7)) return MOE_ERR_INVALID_ARG;
  for (int i = 0; i < count; ++i) {
    const int rc = check(tensors[i]);
    if (rc) return rc;
  }
  if (plan_bytes < moe_adamw_plan_size(tensors, count)) return MOE_ERR_INVALID_ARG;
  Header *h = static_cast<Header *>(plan);
  *h = Header{};
  h->magic = kMagic;
  h->count = count;
  h->chunks_at = (int64_t)(sizeof(Header) + (size_t)count * sizeof(Tensor));
  Tensor *t = reinterpret_cast<Tensor *>(static_cast<uint8_t *>(plan) + sizeof(Header));
  for (int i = 0; i < count; ++i) {
    const moe_adamw_tensor &a = tensors[i];
    const bool f8 = a.state == MOE_ADAMW_F8;
    const uintptr_t wide = reinterpret_cast<uintptr_t>(a.p) | reinterpret_cast<uintptr_t>(a.g) |
                           reinterpret_cast<uintptr_t>(a.master) |
                           (f8 ? 0 : reinterpret_cast<uintptr_t>(a.m) | reinterpret_cast<uintptr_t>(a.v));
    const uintptr_t narrow = f8 ? reinterpret_cast<uintptr_t>(a.m) | reinterpret_cast<uintptr_t>(a.v) : 0;
    t[i] = Tensor{a.p, a.master, a.g, a.m, a.v, a.m_scale, a.v_scale, a.n, a.weight_decay,
                  (wide & 15) == 0 && (narrow & 7) == 0};
  }
  Chunk *c = reinterpret_cast<Chunk *>(static_cast<uint8_t *>(plan) + h->chunks_at);
  for (int k = 0; k < KINDS; ++k) {
    for (int i = 0; i < count; ++i) {
      if (kind_of(tensors[i]) != k) continue;
      const int64_t n = (tensors[i].n + kChunk - 1) / kChunk;
      for (int64_t j = 0; j < n; ++j) *c++ = Chunk{i, (int32_t)j};
      h->chunks[k] += n;
    }
  }
  return MOE_OK;
}

extern "C" int moe_adamw_step(const void *plan_host, const void *plan_device, double beta1, double beta2, float eps,
                              moe_adamw_state *state, moe_stream_t stream) {
  const Header *h = static_cast<const Header *>(plan_host);
  if (!h || h->magic != kMagic || !plan_device || !aligned16(plan_device) || !state ||
      (reinterpret_cast<uintptr_t>(state) & 7))
    return MOE_ERR_INVALID_ARG;
  if (!(beta1 >= 0.0 && beta1 < 1.0) || !(beta2 >= 0.0 && beta2 < 1.0) || !(eps > 0.0f)) return MOE_ERR_INVALID_ARG;
  const Hyper hy{(float)beta1, (float)beta2, (float)(1.0 - beta1), (float)(1.0 - beta2), eps, (float)std::log(beta1),
                 (float)std::log(beta2)};
  const uint8_t *dev = static_cast<const uint8_t *>(plan_device);
  cudaStream_t s = (cudaStream_t)stream;
  int last = 0;   // the launch that advances the step count (an empty plan still counts a step)
  for (int k = 0; k < KINDS; ++k)
    if (h->chunks[k]) last = k;
  int64_t first = 0;
  for (int k = 0; k <= last; ++k) {
    const int64_t n = h->chunks[k];
    if (n == 0 && k != last) continue;
    int rc = MOE_OK;
    switch (k) {
      case F32_F32: rc = launch<F32_F32>(dev, h, first, n, hy, state, k == last, s); break;
      case BF16_F32: rc = launch<BF16_F32>(dev, h, first, n, hy, state, k == last, s); break;
      case BF16_MASTER_F32: rc = launch<BF16_MASTER_F32>(dev, h, first, n, hy, state, k == last, s); break;
      case F32_F8: rc = launch<F32_F8>(dev, h, first, n, hy, state, k == last, s); break;
      case BF16_F8: rc = launch<BF16_F8>(dev, h, first, n, hy, state, k == last, s); break;
      default: rc = launch<BF16_MASTER_F8>(dev, h, first, n, hy, state, k == last, s); break;
    }
    if (rc) return rc;
    first += n;
  }
  return MOE_OK;
}
