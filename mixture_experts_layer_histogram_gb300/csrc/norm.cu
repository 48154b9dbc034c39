// RMS norms before and after a block, fused with the block's gate and the scaled residual, forward
// and backward.
//
//   n   = x rms(x) w                                   rms(v) = 1 / sqrt(mean(v^2) + eps)
//   out = a x + g * (y rms(y) w_post),   n = out rms(out) w_next       g: none, [d] or [T, d]
//
// With r = rms(v), u = dn w, the norm's backward is dv = r (u - v r^2 mean(u v)), dw = sum_t dn v r.
// The backward of the fused form takes G = dout + (norm backward of dn at out), then dx = a G, and
// the norm backward at y with u = g w_post G. It needs mean(u y) before G is known; u is linear in G, so
//   sum u y = sum q dout + r (sum q w_next dn) - r^3 mean(w_next dn out) (sum q out),   q = g w_post y,
// and one reduction of six sums serves the whole row (its rounding error is of the order of the one
// that the subtraction in G makes).
//
// HBM-bound: a thread block works on one row at a time, every row is read once and written once. Rows come
// through a ring of up to three stages in shared memory, filled by cp.async: the copies of the next rows are in
// flight while a row is reduced, whatever the registers hold. Where a row is a multiple of 16 bytes each
// thread copies and reads its own vectors, so no barrier stands between copy and use. Other rows are copied as the
// 16-byte windows that cover them (aligned, whole sectors) and read one element per lane after a barrier.
// Measured (bf16, channel gate, next norm): forward at T = 8192, d = 2048 25.1 us (134 MB, 5.4 TB/s), backward at
// T = 16384, d = 4096 132 us (805 MB, 6.1 TB/s); fp32 rows of 1537 with a token gate, T = 8192, 81 us (403 MB, 5.0 TB/s).
// The norm before a block (bf16, T = 16384, d = 4096): forward 47.3 us (268 MB, 5.7 TB/s), backward with dx_in 90.4 us
// (537 MB, 5.9 TB/s); at T = 8192, d = 2048 14.7 and 28.3 us.
// Before: rows in registers without the ring and one fp32 per instruction took 34 and 288 us, the ring alone 31 and
// 278 us; the instructions were the bound, which pairs of fp32, shared addresses formed once per row and weights
// kept in registers took off.
//
// The weight gradients are summed over a block's rows in registers, written as one fp32 partial row per block and
// added up by a second kernel in a fixed order, so they do not depend on timing. With a gate per
// channel, dw_post and d_gate are both multiples of A = sum_t G y r, so one accumulator serves both.
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

struct FwdParams {
  const void *y, *x, *w_post, *gate, *w_next;
  void *out, *n;
  int64_t T;
  int d, gate_kind;
  float res_scale, eps;
};

// BLOCK: the residual form (out from y, x); without it x itself is normed. NEXT: n is written. With few vectors
// per thread the weights stay in registers from row to row.
template <typename T, int VEC, int ITER, bool BLOCK, bool NEXT>
__global__ void __launch_bounds__(kMaxThreads, ITER == 1 ? 2 : 1) norm_fwd_kernel(const FwdParams p, const Geometry geom) {
  using V = Lanes<T, VEC, float>;
  using L = typename V::L;
  constexpr int N = V::N;
  constexpr bool kHold = ITER * VEC <= 16 && ITER <= 4;
  extern __shared__ __align__(16) uint8_t dyn[];
  __shared__ SumBuf sums;
  const Ring<T, VEC, ITER> ring(dyn, geom, p.T, p.d);
  int half = 0;
  const float inv_d = 1.0f / (float)p.d;
  const bool token = BLOCK && p.gate_kind == MOE_GATE_TOKEN, channel = BLOCK && p.gate_kind == MOE_GATE_CHANNEL;
  clear(sums);
  auto fetch = [&](int64_t row, int stage) {   // x, y, gate
    if (row < p.T) {
      const int64_t off = ring.offset(row);
      ring.fetch(p.x, off, stage, 0);
      if (BLOCK) ring.fetch(p.y, off, stage, 1);
      if (token) ring.fetch(p.gate, off, stage, 2);
    }
    ring.commit();
  };
  for (int s = 0; s < ring.stages - 1; ++s) fetch(blockIdx.x + (int64_t)s * gridDim.x, s);
  // w_post (times the channel gate) and w_next of vector v
  auto weights = [&](int v, L *wg, L *wn) {
    if (BLOCK) {
      V::load((const T *)p.w_post + (int64_t)v * VEC, wg);
      if (channel) {
        L g[N];
        V::load((const T *)p.gate + (int64_t)v * VEC, g);
#pragma unroll
        for (int c = 0; c < N; ++c) wg[c] = mul(wg[c], g[c]);
      }
    }
    if (NEXT) V::load((const T *)p.w_next + (int64_t)v * VEC, wn);
  };
  L hold_g[kHold ? ITER : 1][N], hold_n[kHold ? ITER : 1][N];
  if (kHold) {
#pragma unroll
    for (int i = 0; i < ITER; ++i)
      if (ring.has(i)) weights(threadIdx.x + i * blockDim.x, hold_g[kHold ? i : 0], hold_n[kHold ? i : 0]);
  }
  const L scale = splat<L>(p.res_scale);
  int stage = 0;
  for (int64_t row = blockIdx.x; row < p.T; row += gridDim.x) {
    if (ring.stages == 1) {
      if (VEC == 1) __syncthreads();   // every thread has left the row before
      fetch(row, 0);
    }
    ring.wait();
    const int64_t off = ring.offset(row);
    const uint32_t here = ring.at(stage, off);
    auto place = [&](void *out, int i) {   // of this thread's i-th vector in an output
      return reinterpret_cast<T *>((uint8_t *)out + off + (VEC > 1 ? 0u : (uint32_t)sizeof(T) * threadIdx.x) + i * ring.step);
    };
    L o[ITER][N];
    float r = 0.0f;
    if (BLOCK) {
      L s = splat<L>(0.0f);
#pragma unroll
      for (int i = 0; i < ITER; ++i) {
        if (!ring.has(i)) continue;
        V::load_shared(here + ring.row_bytes + i * ring.step, o[i]);
#pragma unroll
        for (int c = 0; c < N; ++c) s = fma(o[i][c], o[i][c], s);
      }
      r = rsqrtf(block_sum(total(s), sums, half) * inv_d + p.eps);
    }
    L s = splat<L>(0.0f), rr = splat<L>(r);
#pragma unroll
    for (int i = 0; i < ITER; ++i) {
      if (!ring.has(i)) continue;
      const int v = threadIdx.x + i * blockDim.x;
      L x[N];
      V::load_shared(here + i * ring.step, x);
      if (BLOCK) {
        L(&wg)[N] = hold_g[kHold ? i : 0];
        if (!kHold) weights(v, wg, hold_n[0]);
#pragma unroll
        for (int c = 0; c < N; ++c) o[i][c] = mul(mul(o[i][c], rr), wg[c]);
        if (token) {
          L g[N];
          V::load_shared(here + 2 * ring.row_bytes + i * ring.step, g);
#pragma unroll
          for (int c = 0; c < N; ++c) o[i][c] = mul(o[i][c], g[c]);
        }
#pragma unroll
        for (int c = 0; c < N; ++c) o[i][c] = fma(scale, x[c], o[i][c]);
        V::store(place(p.out, i), o[i]);
      } else {
#pragma unroll
        for (int c = 0; c < N; ++c) o[i][c] = x[c];
      }
      if (NEXT) {
#pragma unroll
        for (int c = 0; c < N; ++c) s = fma(o[i][c], o[i][c], s);
      }
    }
    // the row is in registers: its stage's successor may be overwritten (windows: the barrier of wait() has
    // passed, so every thread has left that row)
    if (ring.stages > 1) fetch(row + (int64_t)(ring.stages - 1) * gridDim.x, ring.freed(stage));
    if (NEXT) {   // from the unrounded stream: n is rounded once
      rr = splat<L>(rsqrtf(block_sum(total(s), sums, half) * inv_d + p.eps));
#pragma unroll
      for (int i = 0; i < ITER; ++i) {
        if (!ring.has(i)) continue;
        const int v = threadIdx.x + i * blockDim.x;
        L(&wn)[N] = hold_n[kHold ? i : 0];
        if (!kHold) V::load((const T *)p.w_next + (int64_t)v * VEC, wn);
#pragma unroll
        for (int c = 0; c < N; ++c) o[i][c] = mul(mul(o[i][c], rr), wn[c]);
        V::store(place(p.n, i), o[i]);
      }
    }
    if (++stage == ring.stages) stage = 0;
  }
}

// Blocks of kMaxThreads that the backward's registers leave room for: the accumulators and weights of a 16-byte
// vector per thread take over 64, four single elements do not.
constexpr int bwd_per_sm(int vec, int iter) { return vec == 1 && iter <= 4 ? 2 : 1; }

struct BwdParams {
  const void *dout, *dn, *out, *y, *w_post, *gate, *w_next;   // dout may be null (zero)
  void *dx, *dy, *d_gate;                                     // d_gate here: the [T, d] one
  float *part;                                                // [2][blocks][d]: dw_next, then A (or dw_post)
  int64_t T;
  int d, gate_kind;
  float res_scale, eps;
};

template <int N> __device__ __forceinline__ void put_part(float *p, const F2 (&v)[N]) {
#pragma unroll
  for (int i = 0; i < N; i += 2) *reinterpret_cast<ulonglong2 *>(p + 2 * i) = make_ulonglong2(v[i].v, v[i + 1].v);
}
__device__ __forceinline__ void put_part(float *p, const float (&v)[1]) { *p = v[0]; }
__device__ __forceinline__ void put_part(float *p, const double (&v)[1]) { *p = (float)v[0]; }
__device__ __forceinline__ float inv_root(float v) { return rsqrtf(v); }
__device__ __forceinline__ double inv_root(double v) { return 1.0 / sqrt(v); }

// BLOCK: the residual form; without it the backward of one norm (out = its input, w_next its weights).
// S: the type of the sums and of the differences u - v r^2 mean(u v). In a row of few values the two terms
// can all but cancel (in a row of one value what is left is u eps r^2), so rows of at most 32 values are
// computed in 64 bits; a warp holds such a row at one value per lane.
template <typename T, int VEC, int ITER, bool BLOCK, bool NEXT, typename S>
__global__ void __launch_bounds__(kMaxThreads, bwd_per_sm(VEC, ITER)) norm_bwd_kernel(const BwdParams p, const Geometry geom) {
  using V = Lanes<T, VEC, S>;
  using L = typename V::L;
  constexpr int N = V::N;
  constexpr bool kHold = ITER * VEC <= 16 && ITER <= 4;
  extern __shared__ __align__(16) uint8_t dyn[];
  __shared__ SumBuf sums;
  const Ring<T, VEC, ITER> ring(dyn, geom, p.T, p.d);
  int half = 0;
  const S inv_d = S(1) / (S)p.d;
  const bool has_d = p.dout != nullptr;
  const bool token = BLOCK && p.gate_kind == MOE_GATE_TOKEN, channel = BLOCK && p.gate_kind == MOE_GATE_CHANNEL;
  // buffers of a stage: dn, out, y, then dout and gate where they are
  constexpr int kDn = 0, kOut = NEXT ? 1 : 0, kY = NEXT ? 2 : 0, kFixed = (NEXT ? 2 : 0) + (BLOCK ? 1 : 0);
  const int at_d = kFixed, at_g = kFixed + (has_d ? 1 : 0);
  clear(sums);
  auto fetch = [&](int64_t row, int stage) {
    if (row < p.T) {
      const int64_t off = ring.offset(row);
      if (NEXT) {
        ring.fetch(p.dn, off, stage, kDn);
        ring.fetch(p.out, off, stage, kOut);
      }
      if (BLOCK) ring.fetch(p.y, off, stage, kY);
      if (has_d) ring.fetch(p.dout, off, stage, at_d);
      if (token) ring.fetch(p.gate, off, stage, at_g);
    }
    ring.commit();
  };
  L acc_n[ITER][N], acc_p[ITER][N];
#pragma unroll
  for (int i = 0; i < ITER; ++i) {
#pragma unroll
    for (int c = 0; c < N; ++c) acc_n[i][c] = acc_p[i][c] = splat<L>(0.0f);
  }
  for (int s = 0; s < ring.stages - 1; ++s) fetch(blockIdx.x + (int64_t)s * gridDim.x, s);
  // w_post (times the channel gate) and w_next of vector v
  auto weights = [&](int v, L *wg, L *wn) {
    if (BLOCK) {
      V::load((const T *)p.w_post + (int64_t)v * VEC, wg);
      if (channel) {
        L g[N];
        V::load((const T *)p.gate + (int64_t)v * VEC, g);
#pragma unroll
        for (int c = 0; c < N; ++c) wg[c] = mul(wg[c], g[c]);
      }
    }
    if (NEXT) V::load((const T *)p.w_next + (int64_t)v * VEC, wn);
  };
  L hold_g[kHold ? ITER : 1][N], hold_n[kHold ? ITER : 1][N];
  if (kHold) {
#pragma unroll
    for (int i = 0; i < ITER; ++i)
      if (ring.has(i)) weights(threadIdx.x + i * blockDim.x, hold_g[kHold ? i : 0], hold_n[kHold ? i : 0]);
  }
  int stage = 0;
  for (int64_t row = blockIdx.x; row < p.T; row += gridDim.x) {
    if (ring.stages == 1) {
      if (VEC == 1) __syncthreads();   // every thread has left the row before
      fetch(row, 0);
    }
    ring.wait();
    // every thread has left the row before (its own vectors: the thread itself; windows: the barrier in wait())
    if (ring.stages > 1) fetch(row + (int64_t)(ring.stages - 1) * gridDim.x, ring.freed(stage));
    const int64_t off = ring.offset(row);
    const uint32_t here = ring.at(stage, off);
    auto place = [&](void *out, int i) {   // of this thread's i-th vector in an output
      return reinterpret_cast<T *>((uint8_t *)out + off + (VEC > 1 ? 0u : (uint32_t)sizeof(T) * threadIdx.x) + i * ring.step);
    };
    // out^2, out w_next dn | y^2, q dout, q w_next dn, q out
    L t[6];
#pragma unroll
    for (int i = 0; i < 6; ++i) t[i] = splat<L>(0.0f);
#pragma unroll
    for (int i = 0; i < ITER; ++i) {
      if (!ring.has(i)) continue;
      const int v = threadIdx.x + i * blockDim.x;
      L(&wg)[N] = hold_g[kHold ? i : 0], (&wn)[N] = hold_n[kHold ? i : 0];
      if (!kHold) weights(v, wg, wn);
      L u[N], o[N], q[N];
      if (NEXT) {
        V::load_shared(here + kDn * ring.row_bytes + i * ring.step, u);
        V::load_shared(here + kOut * ring.row_bytes + i * ring.step, o);
#pragma unroll
        for (int c = 0; c < N; ++c) {
          u[c] = mul(u[c], wn[c]);
          t[0] = fma(o[c], o[c], t[0]);
          t[1] = fma(o[c], u[c], t[1]);
        }
      }
      if (BLOCK) {
        V::load_shared(here + kY * ring.row_bytes + i * ring.step, q);
#pragma unroll
        for (int c = 0; c < N; ++c) {
          t[2] = fma(q[c], q[c], t[2]);
          q[c] = mul(q[c], wg[c]);
        }
        if (token) {
          L g[N];
          V::load_shared(here + at_g * ring.row_bytes + i * ring.step, g);
#pragma unroll
          for (int c = 0; c < N; ++c) q[c] = mul(q[c], g[c]);
        }
        if (has_d) {
          L d[N];
          V::load_shared(here + at_d * ring.row_bytes + i * ring.step, d);
#pragma unroll
          for (int c = 0; c < N; ++c) t[3] = fma(q[c], d[c], t[3]);
        }
        if (NEXT) {
#pragma unroll
          for (int c = 0; c < N; ++c) {
            t[4] = fma(q[c], u[c], t[4]);
            t[5] = fma(q[c], o[c], t[5]);
          }
        }
      }
    }
    S s[6];
#pragma unroll
    for (int i = 0; i < 6; ++i) s[i] = total(t[i]);
    block_sum6(s, sums, half);
    const S rn = NEXT ? inv_root(s[0] * inv_d + p.eps) : S(0);
    const S cn = rn * rn * (s[1] * inv_d);                   // r^2 mean(out u)
    const S ry = BLOCK ? inv_root(s[2] * inv_d + p.eps) : S(0);
    const S uy = s[3] + rn * (s[4] - cn * s[5]);             // sum u y
    const S cy = ry * ry * (uy * inv_d);
    const L Rn = all(rn, L()), Cn = all(-cn, L()), Ry = all(ry, L()), Cy = all(-cy, L()), scale = splat<L>(p.res_scale);
#pragma unroll
    for (int i = 0; i < ITER; ++i) {
      if (!ring.has(i)) continue;
      const int v = threadIdx.x + i * blockDim.x;
      L(&wg)[N] = hold_g[kHold ? i : 0], (&wn)[N] = hold_n[kHold ? i : 0];
      if (!kHold) weights(v, wg, wn);
      L G[N], a[N], b[N];
      if (has_d) {
        V::load_shared(here + at_d * ring.row_bytes + i * ring.step, G);
      } else {
#pragma unroll
        for (int c = 0; c < N; ++c) G[c] = splat<L>(0.0f);
      }
      if (NEXT) {
        V::load_shared(here + kDn * ring.row_bytes + i * ring.step, a);
        V::load_shared(here + kOut * ring.row_bytes + i * ring.step, b);
#pragma unroll
        for (int c = 0; c < N; ++c) {
          G[c] = fma(fma(b[c], Cn, mul(a[c], wn[c])), Rn, G[c]);
          acc_n[i][c] = fma(mul(a[c], Rn), b[c], acc_n[i][c]);
        }
      }
#pragma unroll
      for (int c = 0; c < N; ++c) a[c] = BLOCK ? mul(G[c], scale) : G[c];
      V::store(place(p.dx, i), a);
      if (BLOCK) {
        V::load_shared(here + kY * ring.row_bytes + i * ring.step, a);
        if (token) {   // d_gate = G y r w_post; then wg is per token
          V::load_shared(here + at_g * ring.row_bytes + i * ring.step, b);
          L dg[N];
#pragma unroll
          for (int c = 0; c < N; ++c) {
            const L Gy = mul(mul(a[c], Ry), G[c]);
            acc_p[i][c] = fma(b[c], Gy, acc_p[i][c]);
            dg[c] = mul(Gy, wg[c]);
            G[c] = mul(G[c], b[c]);
          }
          V::store(place(p.d_gate, i), dg);
        } else {
#pragma unroll
          for (int c = 0; c < N; ++c) acc_p[i][c] = fma(mul(a[c], Ry), G[c], acc_p[i][c]);
        }
#pragma unroll
        for (int c = 0; c < N; ++c) a[c] = mul(fma(a[c], Cy, mul(wg[c], G[c])), Ry);
        V::store(place(p.dy, i), a);
      }
    }
    if (++stage == ring.stages) stage = 0;
  }
  start_next();   // the kernel that adds up the partial rows
#pragma unroll
  for (int i = 0; i < ITER; ++i) {
    if (!ring.has(i)) continue;
    const int v = threadIdx.x + i * blockDim.x;
    float *dst = p.part + (int64_t)blockIdx.x * p.d + (int64_t)v * VEC;
    if (NEXT) put_part(dst, acc_n[i]);
    if (BLOCK) put_part(dst + (int64_t)gridDim.x * p.d, acc_p[i]);
  }
}

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

// Blocks of the backward on rows of `tensors` inputs: each leaves a partial row, so there are no more than the GPU
// holds at once. (The SMs of a GB300, not of the current device: the workspace's size follows from it, and may be asked
// for anywhere.)
constexpr int kSms = 152;
static int bwd_blocks(int64_t T, const Shape &s, int tensors) {
  int64_t b = kSms * per_sm(s, tensors, bwd_per_sm(s.vec, s.iter) * kMaxThreads);
  if (b > T) b = T;
  return b < 1 ? 1 : (int)b;
}
// The most partial rows that any form's inputs (two to five) lead to.
static int bwd_blocks_most(int64_t T, const Shape &s) {
  int most = 1;
  for (int tensors = 2; tensors <= 5; ++tensors) {
    const int b = bwd_blocks(T, s, tensors);
    if (b > most) most = b;
  }
  return most;
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
template <typename T, int VEC, int ITER>
static int launch_fwd(const FwdParams &p, bool block, bool next, const Shape &sh, cudaStream_t s) {
  const int tensors = block ? (p.gate_kind == MOE_GATE_TOKEN ? 3 : 2) : 1;
  int64_t grid = (int64_t)sm_count() * per_sm(sh, tensors, sh.iter == 1 ? 2 * kMaxThreads : kMaxThreads);
  if (grid > p.T) grid = p.T;
  if (!block) return launch<norm_fwd_kernel<T, VEC, ITER, false, true>>(p, sh, tensors, (int)grid, s);
  if (next) return launch<norm_fwd_kernel<T, VEC, ITER, true, true>>(p, sh, tensors, (int)grid, s);
  return launch<norm_fwd_kernel<T, VEC, ITER, true, false>>(p, sh, tensors, (int)grid, s);
}
template <typename T, int VEC, int ITER, typename S = float>
static int launch_bwd(const BwdParams &p, bool block, bool next, const Shape &sh, int tensors, int grid, cudaStream_t s) {
  if (!block) return launch<norm_bwd_kernel<T, VEC, ITER, false, true, S>>(p, sh, tensors, grid, s);
  if (next) return launch<norm_bwd_kernel<T, VEC, ITER, true, true, S>>(p, sh, tensors, grid, s);
  return launch<norm_bwd_kernel<T, VEC, ITER, true, false, S>>(p, sh, tensors, grid, s);
}

#define MOE_NORM_DISPATCH(FN, ...)                                                   \
  do {                                                                               \
    if (dtype == MOE_BF16) {                                                         \
      if (sh.vec == 8 && sh.iter == 1) rc = FN<__nv_bfloat16, 8, 1>(__VA_ARGS__);    \
      else if (sh.vec == 8) rc = FN<__nv_bfloat16, 8, 2>(__VA_ARGS__);               \
      else if (sh.iter == 4) rc = FN<__nv_bfloat16, 1, 4>(__VA_ARGS__);              \
      else rc = FN<__nv_bfloat16, 1, 16>(__VA_ARGS__);                               \
    } else {                                                                         \
      if (sh.vec == 4 && sh.iter == 1) rc = FN<float, 4, 1>(__VA_ARGS__);            \
      else if (sh.vec == 4 && sh.iter == 2) rc = FN<float, 4, 2>(__VA_ARGS__);       \
      else if (sh.vec == 4) rc = FN<float, 4, 4>(__VA_ARGS__);                       \
      else if (sh.iter == 4) rc = FN<float, 1, 4>(__VA_ARGS__);                      \
      else rc = FN<float, 1, 16>(__VA_ARGS__);                                       \
    }                                                                                \
  } while (0)

static int check_shape(int T, int d, int dtype, float eps) {
  if (T < 0 || d < 1 || (dtype != MOE_F32 && dtype != MOE_BF16) || !(eps > 0.0f)) return MOE_ERR_INVALID_ARG;
  if (d > MOE_NORM_MAX_D) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}
static bool bad(const void *p) { return !p || !aligned16(p); }

static int run_fwd(const FwdParams &p, int dtype, bool block, bool next, cudaStream_t s) {
  const Shape sh = shape_of(p.d, dtype);
  int rc = MOE_OK;
  MOE_NORM_DISPATCH(launch_fwd, p, block, next, sh, s);
  return rc;
}

static int run_bwd(BwdParams p, int dtype, bool block, bool next, void *dw_next, void *dw_post, void *d_gate, void *ws,
                   size_t ws_bytes, cudaStream_t s) {
  const Shape sh = shape_of(p.d, dtype);
  const int tensors = (next ? 2 : 0) + (block ? 1 : 0) + (p.dout ? 1 : 0) + (block && p.gate_kind == MOE_GATE_TOKEN ? 1 : 0);
  const int grid = bwd_blocks(p.T, sh, tensors);
  if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255) || ws_bytes < moe_norm_bwd_workspace_size((int)p.T, p.d, dtype))
    return MOE_ERR_INVALID_ARG;
  p.part = static_cast<float *>(ws);
  int rc = MOE_OK;
  if (p.d <= 32) {   // one element per lane, in 64 bits
    Shape one = sh;
    one.vec = one.iter = 1;
    one.threads = 32;
    one.row_bytes = ((uint32_t)p.d * (uint32_t)dtype_size(dtype) + 15) / 16 * 16 + 16;
    if (dtype == MOE_BF16) rc = launch_bwd<__nv_bfloat16, 1, 1, double>(p, block, next, one, tensors, grid, s);
    else rc = launch_bwd<float, 1, 1, double>(p, block, next, one, tensors, grid, s);
  } else {
    MOE_NORM_DISPATCH(launch_bwd, p, block, next, sh, tensors, grid, s);
  }
  if (rc) return rc;
  const dim3 g((p.d + 31) / 32, block ? 2 : 1);
  if (dtype == MOE_BF16) {
    using B = __nv_bfloat16;
    MOE_TRY_CUDA(launch_after(norm_bwd_sum_kernel<B>, g, dim3(1024), 0, s, p.part, grid, p.d, p.gate_kind,
                              (const B *)p.w_post, (const B *)p.gate, (B *)dw_next, (B *)dw_post, (B *)d_gate));
  } else {
    MOE_TRY_CUDA(launch_after(norm_bwd_sum_kernel<float>, g, dim3(1024), 0, s, p.part, grid, p.d, p.gate_kind,
                              (const float *)p.w_post, (const float *)p.gate, (float *)dw_next, (float *)dw_post,
                              (float *)d_gate));
  }
  return MOE_OK;
}

}  // namespace norm
}  // namespace moe

using namespace moe;
using namespace moe::norm;

extern "C" size_t moe_norm_bwd_workspace_size(int T, int d, int dtype) {
  if (T < 0 || d < 1) return 0;
  return (size_t)2 * bwd_blocks_most(T, shape_of(d, dtype)) * d * sizeof(float) + 256;
}

extern "C" int moe_norm_fwd(const void *x, const void *w, int T, int d, int dtype, float eps, void *n,
                            moe_stream_t stream) {
  int rc = check_shape(T, d, dtype, eps);
  if (rc) return rc;
  if (T == 0) return MOE_OK;
  if (bad(x) || bad(w) || bad(n)) return MOE_ERR_INVALID_ARG;
  FwdParams p{};
  p.x = x;
  p.w_next = w;
  p.n = n;
  p.T = T;
  p.d = d;
  p.eps = eps;
  return run_fwd(p, dtype, false, true, (cudaStream_t)stream);
}

extern "C" int moe_norm_residual_fwd(const void *y, const void *x, const void *w_post, const void *gate, int gate_kind,
                                     const void *w_next, int T, int d, int dtype, float res_scale, float eps, void *out,
                                     void *n, moe_stream_t stream) {
  int rc = check_shape(T, d, dtype, eps);
  if (rc) return rc;
  if (gate_kind < MOE_GATE_NONE || gate_kind > MOE_GATE_TOKEN) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  if (!w_next && n) return MOE_ERR_INVALID_ARG;
  if (bad(y) || bad(x) || bad(w_post) || bad(out) || (gate_kind != MOE_GATE_NONE && bad(gate)) ||
      (w_next && (bad(w_next) || bad(n))))
    return MOE_ERR_INVALID_ARG;
  FwdParams p{};
  p.y = y;
  p.x = x;
  p.w_post = w_post;
  p.gate = gate;
  p.gate_kind = gate_kind;
  p.w_next = w_next;
  p.out = out;
  p.n = n;
  p.T = T;
  p.d = d;
  p.res_scale = res_scale;
  p.eps = eps;
  return run_fwd(p, dtype, true, w_next != nullptr, (cudaStream_t)stream);
}

extern "C" int moe_norm_bwd(const void *dn, const void *x, const void *w, const void *dx_in, int T, int d, int dtype,
                            float eps, void *dx, void *dw, void *ws, size_t ws_bytes, moe_stream_t stream) {
  int rc = check_shape(T, d, dtype, eps);
  if (rc) return rc;
  if (bad(dw) || bad(w) || (T > 0 && (bad(dn) || bad(x) || bad(dx) || (dx_in && bad(dx_in))))) return MOE_ERR_INVALID_ARG;
  BwdParams p{};
  p.dout = dx_in;
  p.dn = dn;
  p.out = x;
  p.w_next = w;
  p.dx = dx;
  p.T = T;
  p.d = d;
  p.eps = eps;
  return run_bwd(p, dtype, false, true, dw, nullptr, nullptr, ws, ws_bytes, (cudaStream_t)stream);
}

extern "C" int moe_norm_residual_bwd(const void *dout, const void *dn, const void *out, const void *y,
                                     const void *w_post, const void *gate, int gate_kind, const void *w_next, int T,
                                     int d, int dtype, float res_scale, float eps, void *dx, void *dy, void *dw_post,
                                     void *d_gate, void *dw_next, void *ws, size_t ws_bytes, moe_stream_t stream) {
  int rc = check_shape(T, d, dtype, eps);
  if (rc) return rc;
  if (gate_kind < MOE_GATE_NONE || gate_kind > MOE_GATE_TOKEN || (dn && !w_next)) return MOE_ERR_INVALID_ARG;
  const bool gated = gate_kind != MOE_GATE_NONE;
  if (bad(dw_post) || bad(w_post) || (gated && bad(gate)) || (gate_kind == MOE_GATE_CHANNEL && bad(d_gate)) ||
      (w_next && (bad(w_next) || bad(dw_next))))
    return MOE_ERR_INVALID_ARG;
  if (T > 0 && (((dout || !w_next) && bad(dout)) || (w_next && (bad(dn) || bad(out))) || bad(y) || bad(dx) || bad(dy) ||
                (gate_kind == MOE_GATE_TOKEN && bad(d_gate))))
    return MOE_ERR_INVALID_ARG;
  BwdParams p{};
  p.dout = dout;
  p.dn = dn;
  p.out = out;
  p.y = y;
  p.w_post = w_post;
  p.gate = gate;
  p.gate_kind = gate_kind;
  p.w_next = w_next;
  p.dx = dx;
  p.dy = dy;
  p.d_gate = d_gate;
  p.T = T;
  p.d = d;
  p.res_scale = res_scale;
  p.eps = eps;
  return run_bwd(p, dtype, true, w_next != nullptr, dw_next, dw_post,
                 gate_kind == MOE_GATE_CHANNEL ? d_gate : nullptr, ws, ws_bytes, (cudaStream_t)stream);
}
