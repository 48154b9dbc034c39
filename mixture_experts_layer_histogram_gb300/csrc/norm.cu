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
#include "row_ring.cuh"

namespace moe {
namespace norm {

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
