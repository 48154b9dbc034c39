// What the kernels that work on whole rows share (norm.cu, layer_norm.cu): arithmetic on two values at a time, the ring of
// rows in shared memory, sums over a block, the partial rows of weight gradients and their reduction, launch shapes.
#pragma once

#include <atomic>

#include "common.cuh"
#include "dependent.cuh"
#include "f32x2.cuh"

namespace moe {
namespace norm {

constexpr int kMaxThreads = 512;
constexpr int kMaxWarps = kMaxThreads / 32;
constexpr int kStages = 3;                    // at most; fewer where long rows leave no room
constexpr size_t kRingMost = 200 * 1024;      // bytes; one stage of five fp32 rows of MOE_NORM_MAX_D is 164 KB
static_assert(5 * (MOE_NORM_MAX_D * 4 + 16) <= kRingMost, "every ring fits the limit that launches raise");

// Arithmetic on one lane of values: two fp32 at a time (f32x2 instructions) for rows of 16-byte vectors, one fp32,
// or one fp64. At bf16 the instructions, not HBM, bound these kernels when each value takes its own.
using moe::add;
using moe::fma;
using moe::mul;
template <typename S> __device__ __forceinline__ S mul(S a, S b) { return a * b; }
template <typename S> __device__ __forceinline__ S add(S a, S b) { return a + b; }
__device__ __forceinline__ float fma(float a, float b, float c) { return fmaf(a, b, c); }
__device__ __forceinline__ double fma(double a, double b, double c) { return ::fma(a, b, c); }
template <typename L> __device__ __forceinline__ L splat(float v);
template <> __device__ __forceinline__ F2 splat<F2>(float v) { return pair(v, v); }
template <> __device__ __forceinline__ float splat<float>(float v) { return v; }
template <> __device__ __forceinline__ double splat<double>(float v) { return v; }
__device__ __forceinline__ F2 all(float v, F2) { return pair(v, v); }
__device__ __forceinline__ float all(float v, float) { return v; }
__device__ __forceinline__ double all(double v, double) { return v; }
__device__ __forceinline__ float total(F2 a) {
  float x, y;
  split(a, x, y);
  return x + y;
}
__device__ __forceinline__ float total(float a) { return a; }
__device__ __forceinline__ double total(double a) { return a; }

__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 q;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(q.x), "=r"(q.y), "=r"(q.z), "=r"(q.w) : "r"(a) : "memory");
  return q;
}

// How VEC elements of type T are held: N lanes of type L.
template <typename T, int VEC, typename S> struct Lanes;
template <> struct Lanes<__nv_bfloat16, 8, float> {
  typedef F2 L;
  static constexpr int N = 4;
  static __device__ __forceinline__ void load(const void *p, L *v) {
    unpack(*reinterpret_cast<const uint4 *>(p), v);
  }
  static __device__ __forceinline__ void load_shared(uint32_t a, L *v) { unpack(lds128(a), v); }
  static __device__ __forceinline__ void unpack(const uint4 &q, L *v) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = pair(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
  }
  static __device__ __forceinline__ void store(__nv_bfloat16 *p, const L *v) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float x, y;
      split(v[i], x, y);
      w[i] = pack_bf16x2(x, y);
    }
    *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <> struct Lanes<float, 4, float> {
  typedef F2 L;
  static constexpr int N = 2;
  static __device__ __forceinline__ void load(const void *p, L *v) {
    const ulonglong2 q = *reinterpret_cast<const ulonglong2 *>(p);
    v[0].v = q.x;
    v[1].v = q.y;
  }
  static __device__ __forceinline__ void load_shared(uint32_t a, L *v) {
    asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];" : "=l"(v[0].v), "=l"(v[1].v) : "r"(a) : "memory");
  }
  static __device__ __forceinline__ void store(float *p, const L *v) {
    *reinterpret_cast<ulonglong2 *>(p) = make_ulonglong2(v[0].v, v[1].v);
  }
};
template <typename S> struct Lanes<float, 1, S> {
  typedef S L;
  static constexpr int N = 1;
  static __device__ __forceinline__ void load(const void *p, L *v) { v[0] = *reinterpret_cast<const float *>(p); }
  static __device__ __forceinline__ void load_shared(uint32_t a, L *v) {
    float f;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(f) : "r"(a) : "memory");
    v[0] = f;
  }
  static __device__ __forceinline__ void store(float *p, const L *v) { *p = (float)v[0]; }
};
template <typename S> struct Lanes<__nv_bfloat16, 1, S> {
  typedef S L;
  static constexpr int N = 1;
  static __device__ __forceinline__ void load(const void *p, L *v) {
    v[0] = __bfloat162float(*reinterpret_cast<const __nv_bfloat16 *>(p));
  }
  static __device__ __forceinline__ void load_shared(uint32_t a, L *v) {
    uint16_t h;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(h) : "r"(a) : "memory");
    v[0] = __uint_as_float((uint32_t)h << 16);
  }
  static __device__ __forceinline__ void store(__nv_bfloat16 *p, const L *v) { *p = __float2bfloat16_rn((float)v[0]); }
};

// Geometry of the ring of rows. A stage holds the row buffers of the kernel's tensors, `row_bytes` each. VEC > 1: the
// vector v of a row lies at 16 v of its buffer, where the thread that uses it has copied it to. VEC == 1: the buffer
// holds the 16-byte windows that cover the row, whose first element is then `shift` elements into the first.
struct Geometry {
  uint32_t row_bytes, stage_bytes;
  int stages;
};
// One thread's view of it. ITER: vectors (elements) per thread, blockDim apart.
template <typename T, int VEC, int ITER> struct Ring {
  uint32_t mine;           // shared address of this thread's first vector (VEC == 1: of the ring)
  uint32_t row_bytes, stage_bytes, step;
  int stages, d, nvec;
  int64_t all;             // bytes of one tensor

  __device__ __forceinline__ Ring(const uint8_t *smem, const Geometry &g, int64_t rows, int d_)
      : row_bytes(g.row_bytes), stage_bytes(g.stage_bytes), stages(g.stages), d(d_), nvec(d_ / VEC) {
    mine = (uint32_t)__cvta_generic_to_shared(smem) + (VEC > 1 ? 16u * threadIdx.x : 0u);
    step = VEC > 1 ? 16u * blockDim.x : (uint32_t)sizeof(T) * blockDim.x;
    all = rows * d * (int64_t)sizeof(T);
  }
  // Whether this thread's i-th vector exists
  __device__ __forceinline__ bool has(int i) const { return (int)(threadIdx.x + i * blockDim.x) < nvec; }
  // Byte offset of `row` in a tensor, with the thread's first vector where threads copy their own
  __device__ __forceinline__ int64_t offset(int64_t row) const {
    return row * d * (int64_t)sizeof(T) + (VEC > 1 ? 16u * threadIdx.x : 0u);
  }
  // Copy (asynchronously) the row at `off` (offset()) of one tensor into buffer `slot` of `stage`.
  __device__ __forceinline__ void fetch(const void *base, int64_t off, int stage, int slot) const {
    const uint32_t dst = mine + (uint32_t)stage * stage_bytes + (uint32_t)slot * row_bytes;
    const uint8_t *src = (const uint8_t *)base + off;
    if (VEC > 1) {
#pragma unroll
      for (int i = 0; i < ITER; ++i) {
        if (has(i))
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst + i * step), "l"(src + i * step) : "memory");
      }
    } else {
      const int lead = (int)(off & 15), bytes = lead + d * (int)sizeof(T);
      const int64_t left = all - (off - lead);            // up to the tensor's end
      for (int c = 16 * threadIdx.x; c < bytes; c += 16 * blockDim.x) {
        const int n = left - c < 16 ? (int)(left - c) : 16;   // nothing past the tensor is read
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + c), "l"(src - lead + c), "r"(n) : "memory");
      }
    }
  }
  static __device__ __forceinline__ void commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
  // The oldest row's copies have landed (and are visible to all threads that read them); with three stages the
  // next row's may be in flight.
  __device__ __forceinline__ void wait() const {
    if (stages == 3) asm volatile("cp.async.wait_group 1;" ::: "memory");
    else asm volatile("cp.async.wait_group 0;" ::: "memory");
    if (VEC == 1) __syncthreads();
  }
  // Shared address of this thread's first vector (element) of the row at `off` in `stage`; buffers are row_bytes
  // apart, the thread's vectors `step`.
  __device__ __forceinline__ uint32_t at(int stage, int64_t off) const {
    return mine + (uint32_t)stage * stage_bytes +
           (VEC > 1 ? 0u : ((uint32_t)(off & 15) + (uint32_t)sizeof(T) * threadIdx.x));
  }
  // The stage whose row was the last one before `stage`'s: free once every thread has left that row.
  __device__ __forceinline__ int freed(int stage) const { return stage >= 1 ? stage - 1 : stages - 1; }
};

// Sums over the block, the same on every thread. `buf` alternates between two halves, so one barrier per
// reduction is enough: a half is written again only after the next reduction's barrier.
struct alignas(16) SumBuf {
  float v[2][8][kMaxWarps];
};
static_assert(alignof(SumBuf) >= alignof(float4) && kMaxWarps % 4 == 0, "the sums read it four values at a time");
__device__ __forceinline__ void clear(SumBuf &buf) {   // the places of warps that the block does not have stay 0
  for (int i = threadIdx.x; i < 2 * 8 * kMaxWarps; i += blockDim.x) (&buf.v[0][0][0])[i] = 0.0f;
  __syncthreads();
}
__device__ __forceinline__ float block_sum(float v, SumBuf &buf, int &half) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  if (blockDim.x == 32) return v;
  float *b = buf.v[half][0];
  half ^= 1;
  if ((threadIdx.x & 31) == 0) b[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0.0f;
#pragma unroll
  for (int i = 0; i < kMaxWarps / 4; ++i) {
    if (i * 128 >= (int)blockDim.x) break;
    const float4 q = reinterpret_cast<const float4 *>(b)[i];
    v += (q.x + q.y) + (q.z + q.w);
  }
  return v;
}
// Six sums. In the warp, each exchange halves the values a lane carries (9 exchanges, not 30): lane 4 i ends with value i.
__device__ __forceinline__ void block_sum6(float (&s)[6], SumBuf &buf, int &half) {
  const int lane = threadIdx.x & 31;
  float v[8] = {s[0], s[1], s[2], s[3], s[4], s[5], 0.0f, 0.0f};
#pragma unroll
  for (int n = 4, off = 16; n >= 1; n >>= 1, off >>= 1) {
    const bool up = lane & off;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const float give = up ? v[i] : v[i + n], keep = up ? v[i + n] : v[i];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, give, off);
    }
  }
  float r = v[0];
  r += __shfl_xor_sync(0xffffffffu, r, 2);
  r += __shfl_xor_sync(0xffffffffu, r, 1);
  if (blockDim.x > 32) {
    float(*b)[kMaxWarps] = buf.v[half];
    half ^= 1;
    if ((lane & 3) == 0) b[lane >> 2][threadIdx.x >> 5] = r;
    __syncthreads();
    const float4 q = *reinterpret_cast<const float4 *>(&b[lane >> 2][4 * (lane & 3)]);
    r = (q.x + q.y) + (q.z + q.w);
    r += __shfl_xor_sync(0xffffffffu, r, 1);
    r += __shfl_xor_sync(0xffffffffu, r, 2);
  }
#pragma unroll
  for (int i = 0; i < 6; ++i) s[i] = __shfl_sync(0xffffffffu, r, 4 * i);
}
__device__ __forceinline__ void block_sum6(double (&s)[6], SumBuf &, int &) {   // rows of at most 32 values: one warp
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
#pragma unroll
    for (int i = 0; i < 6; ++i) s[i] += __shfl_xor_sync(0xffffffffu, s[i], off);
  }
}

// One block's partial row of a weight gradient
template <int N> __device__ __forceinline__ void put_part(float *p, const F2 (&v)[N]) {
#pragma unroll
  for (int i = 0; i < N; i += 2) *reinterpret_cast<ulonglong2 *>(p + 2 * i) = make_ulonglong2(v[i].v, v[i + 1].v);
}
__device__ __forceinline__ void put_part(float *p, const float (&v)[1]) { *p = v[0]; }
__device__ __forceinline__ void put_part(float *p, const double (&v)[1]) { *p = (float)v[0]; }

// Column sums of the blocks' partial rows, in a fixed order: 32 columns and 32 row groups per block.
template <typename T>
__global__ void __launch_bounds__(1024) norm_bwd_sum_kernel(const float *part, int blocks, int d, int gate_kind,
                                                            const T *w_post, const T *gate, T *dw_next, T *dw_post,
                                                            T *d_gate) {
  wait_previous();
  __shared__ float s[32][33];
  const int lane = threadIdx.x & 31, grp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  const bool second = blockIdx.y != 0;   // 0: dw_next, 1: A
  if ((second && !dw_post) || (!second && !dw_next)) return;
  const float *src = part + (second ? (int64_t)blocks * d : 0);
  float a = 0.0f;
  if (c < d) {
#pragma unroll 8
    for (int b = grp; b < blocks; b += 32) a += src[(int64_t)b * d + c];
  }
  s[grp][lane] = a;
  __syncthreads();
  if (grp != 0 || c >= d) return;
  a = 0.0f;
#pragma unroll
  for (int i = 0; i < 32; ++i) a += s[i][lane];
  auto put = [](T *dst, float v) {
    if constexpr (sizeof(T) == 4) *dst = v;
    else *dst = __float2bfloat16_rn(v);
  };
  if (!second) {
    put(dw_next + c, a);
  } else if (gate_kind == MOE_GATE_CHANNEL) {
    put(dw_post + c, a * (float)gate[c]);
    put(d_gate + c, a * (float)w_post[c]);
  } else {
    put(dw_post + c, a);
  }
}

// Geometry of one row length: 16-byte vectors where a row is a multiple of 16 bytes, else single elements; values per
// thread (iter vectors) and threads per block; the ring's row buffers.
struct Shape {
  int vec, iter, threads;
  uint32_t row_bytes;
};
static Shape shape_of(int d, int dtype) {
  const int es = dtype == MOE_BF16 ? 2 : 4, full = 16 / es;
  Shape s;
  s.vec = d % full == 0 ? full : 1;
  const int nvec = d / s.vec;
  s.iter = s.vec > 1 ? 1 : 4;
  while (s.iter * kMaxThreads < nvec) s.iter *= s.vec > 1 ? 2 : 4;
  s.threads = ((nvec + s.iter - 1) / s.iter + 31) / 32 * 32;
  s.row_bytes = s.vec > 1 ? (uint32_t)d * es : ((uint32_t)d * es + 15) / 16 * 16 + 16;   // windows may start 15 bytes early
  return s;
}
static int stages_of(const Shape &s, int tensors) {
  int n = kStages;
  while (n > 1 && (size_t)n * tensors * s.row_bytes > kRingMost) --n;
  return n;
}
static size_t ring_bytes(const Shape &s, int tensors) { return (size_t)stages_of(s, tensors) * tensors * s.row_bytes; }

// Blocks that an SM holds at once, by threads (the kernels' launch bounds) and by shared memory.
static int per_sm(const Shape &s, int tensors, int threads_max) {
  int n = threads_max / s.threads;
  const int by_smem = (int)((size_t)220 * 1024 / (ring_bytes(s, tensors) + 2048));
  if (n > by_smem) n = by_smem;
  return n < 1 ? 1 : (n > 16 ? 16 : n);
}

// A kernel's dynamic shared memory limit is raised to the largest ring once per device, whatever this call needs: it is
// the process's, and another thread may launch the same kernel on rows of another length at any time.
template <auto KERNEL> static int raise_limit() {
  static std::atomic<uint64_t> raised{0};
  int dev = 0;
  MOE_TRY_CUDA(cudaGetDevice(&dev));
  if (dev < 64 && (raised.load(std::memory_order_relaxed) >> dev & 1)) return MOE_OK;
  MOE_TRY_CUDA(cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kRingMost));
  if (dev < 64) raised.fetch_or((uint64_t)1 << dev, std::memory_order_relaxed);
  return MOE_OK;
}

template <auto KERNEL, typename Params>
static int launch(const Params &p, const Shape &sh, int tensors, int grid, cudaStream_t s) {
  const size_t smem = ring_bytes(sh, tensors);
  const Geometry ring{sh.row_bytes, tensors * sh.row_bytes, stages_of(sh, tensors)};
  if (smem > 40 * 1024) {   // with the sums' buffer past the 48 KB that every kernel may have
    const int rc = raise_limit<KERNEL>();
    if (rc) return rc;
  }
  KERNEL<<<grid, sh.threads, smem, s>>>(p, ring);
  MOE_CHECK_LAUNCH();
  return MOE_OK;
}
static int check_shape(int T, int d, int dtype, float eps) {
  if (T < 0 || d < 1 || (dtype != MOE_F32 && dtype != MOE_BF16) || !(eps > 0.0f)) return MOE_ERR_INVALID_ARG;
  if (d > MOE_NORM_MAX_D) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}
static bool bad(const void *p) { return !p || !aligned16(p); }

}  // namespace norm
}  // namespace moe
