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
// One thread block per row, the row in registers (read once, written once); HBM-bound. The weight
// gradients are summed over a block's rows in registers, written as one fp32 partial row per block and
// added up by a second kernel in a fixed order, so they do not depend on timing. With a gate per
// channel, dw_post and d_gate are both multiples of A = sum_t G y r, so one accumulator serves both.
#include "common.cuh"

namespace moe {
namespace norm {

constexpr int kMaxThreads = 512;
constexpr int kSums = 8;   // floats per warp in the reduction buffer

// VEC elements of type T as they lie in memory: a 16-byte vector, or one element for rows whose
// length is no multiple of 16 bytes.
template <typename T, int VEC> struct Pack;
template <> struct Pack<float, 4> {
  uint4 q;
  __device__ __forceinline__ void load(const float *p) { q = *reinterpret_cast<const uint4 *>(p); }
  __device__ __forceinline__ void load_once(const float *p) { q = ld_stream(reinterpret_cast<const uint4 *>(p)); }
  __device__ __forceinline__ void unpack(float *v) const {
    v[0] = __uint_as_float(q.x); v[1] = __uint_as_float(q.y); v[2] = __uint_as_float(q.z); v[3] = __uint_as_float(q.w);
  }
  static __device__ __forceinline__ void store(float *p, const float *v) {
    *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
  }
};
template <> struct Pack<__nv_bfloat16, 8> {
  uint4 q;
  __device__ __forceinline__ void load(const __nv_bfloat16 *p) { q = *reinterpret_cast<const uint4 *>(p); }
  __device__ __forceinline__ void load_once(const __nv_bfloat16 *p) { q = ld_stream(reinterpret_cast<const uint4 *>(p)); }
  __device__ __forceinline__ void unpack(float *v) const { unpack_bf16x8(q, v); }
  static __device__ __forceinline__ void store(__nv_bfloat16 *p, const float *v) {
    *reinterpret_cast<uint4 *>(p) = pack_bf16x8(v);
  }
};
template <> struct Pack<float, 1> {
  float q;
  __device__ __forceinline__ void load(const float *p) { q = *p; }
  __device__ __forceinline__ void load_once(const float *p) { q = *p; }
  __device__ __forceinline__ void unpack(float *v) const { v[0] = q; }
  static __device__ __forceinline__ void store(float *p, const float *v) { *p = v[0]; }
};
template <> struct Pack<__nv_bfloat16, 1> {
  __nv_bfloat16 q;
  __device__ __forceinline__ void load(const __nv_bfloat16 *p) { q = *p; }
  __device__ __forceinline__ void load_once(const __nv_bfloat16 *p) { q = *p; }
  __device__ __forceinline__ void unpack(float *v) const { v[0] = __bfloat162float(q); }
  static __device__ __forceinline__ void store(__nv_bfloat16 *p, const float *v) { *p = __float2bfloat16_rn(v[0]); }
};

// Sums of N values over the block, the same on every thread. `buf` alternates between two halves, so
// one barrier per reduction is enough: a half is written again only after the next reduction's barrier.
template <int N, typename S>
__device__ __forceinline__ void block_sum(S (&v)[N], float *buf, int &half) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], off);
  }
  const int nw = blockDim.x >> 5;
  if (nw == 1) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float *b = buf + half * (kMaxThreads / 32) * kSums;
  half ^= 1;
  if (lane == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) b[warp * kSums + i] = v[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = lane < nw ? b[lane * kSums + i] : 0.0f;
#pragma unroll
  for (int off = kMaxThreads / 64; off > 0; off >>= 1) {   // nw <= 16: lanes 0..15 hold the warps' sums
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], off);
  }
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = __shfl_sync(0xffffffffu, v[i], 0);
}

struct FwdParams {
  const void *y, *x, *w_post, *gate, *w_next;
  void *out, *n;
  int64_t T;
  int d, gate_kind;
  float res_scale, eps;
};

// BLOCK: the residual form (out from y, x); without it x itself is normed. NEXT: n is written.
template <typename T, int VEC, int ITER, bool BLOCK, bool NEXT>
__global__ void __launch_bounds__(kMaxThreads) norm_fwd_kernel(const FwdParams p) {
  using P = Pack<T, VEC>;
  __shared__ float buf[2 * (kMaxThreads / 32) * kSums];
  int half = 0;
  const int nvec = p.d / VEC;
  const float inv_d = 1.0f / (float)p.d;
  for (int64_t row = blockIdx.x; row < p.T; row += gridDim.x) {
    const int64_t base = row * p.d;
    P px[ITER], py[ITER];
#pragma unroll
    for (int i = 0; i < ITER; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      if (v >= nvec) continue;
      px[i].load_once((const T *)p.x + base + (int64_t)v * VEC);
      if (BLOCK) py[i].load_once((const T *)p.y + base + (int64_t)v * VEC);
    }
    float o[ITER][VEC];
    if (BLOCK) {
      float s[1] = {0.0f};
#pragma unroll
      for (int i = 0; i < ITER; ++i) {
        const int v = threadIdx.x + i * blockDim.x;
        if (v >= nvec) continue;
        float t[VEC];
        py[i].unpack(t);
#pragma unroll
        for (int c = 0; c < VEC; ++c) s[0] = fmaf(t[c], t[c], s[0]);
      }
      block_sum(s, buf, half);
      const float r = 1.0f / sqrtf(s[0] * inv_d + p.eps);
#pragma unroll
      for (int i = 0; i < ITER; ++i) {
        const int v = threadIdx.x + i * blockDim.x;
        if (v >= nvec) continue;
        float ty[VEC], tx[VEC], tw[VEC], tg[VEC];
        P pw, pg;
        pw.load((const T *)p.w_post + (int64_t)v * VEC);
        pw.unpack(tw);
        if (p.gate_kind != MOE_GATE_NONE) {
          pg.load((const T *)p.gate + (p.gate_kind == MOE_GATE_TOKEN ? base : 0) + (int64_t)v * VEC);
          pg.unpack(tg);
#pragma unroll
          for (int c = 0; c < VEC; ++c) tw[c] *= tg[c];
        }
        py[i].unpack(ty);
        px[i].unpack(tx);
#pragma unroll
        for (int c = 0; c < VEC; ++c) o[i][c] = fmaf(p.res_scale, tx[c], ty[c] * r * tw[c]);
        P::store((T *)p.out + base + (int64_t)v * VEC, o[i]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < ITER; ++i) {
        if ((int)(threadIdx.x + i * blockDim.x) < nvec) px[i].unpack(o[i]);
      }
    }
    if (NEXT) {   // from the unrounded stream: n is rounded once
      float s[1] = {0.0f};
#pragma unroll
      for (int i = 0; i < ITER; ++i) {
        if ((int)(threadIdx.x + i * blockDim.x) >= nvec) continue;
#pragma unroll
        for (int c = 0; c < VEC; ++c) s[0] = fmaf(o[i][c], o[i][c], s[0]);
      }
      block_sum(s, buf, half);
      const float r = 1.0f / sqrtf(s[0] * inv_d + p.eps);
#pragma unroll
      for (int i = 0; i < ITER; ++i) {
        const int v = threadIdx.x + i * blockDim.x;
        if (v >= nvec) continue;
        float tw[VEC], t[VEC];
        P pw;
        pw.load((const T *)p.w_next + (int64_t)v * VEC);
        pw.unpack(tw);
#pragma unroll
        for (int c = 0; c < VEC; ++c) t[c] = o[i][c] * r * tw[c];
        P::store((T *)p.n + base + (int64_t)v * VEC, t);
      }
    }
  }
}

struct BwdParams {
  const void *dout, *dn, *out, *y, *w_post, *gate, *w_next;   // dout may be null (zero)
  void *dx, *dy, *d_gate;                                     // d_gate here: the [T, d] one
  float *part;                                                // [2][blocks][d]: dw_next, then A (or dw_post)
  int64_t T;
  int d, gate_kind;
  float res_scale, eps;
};

// BLOCK: the residual form; without it the backward of one norm (out = its input, w_next its weights).
// S: the type of the sums and of the differences u - v r^2 mean(u v). In a row of few values the two terms
// can all but cancel (in a row of one value what is left is u eps r^2), so rows of at most 32 values are
// computed in 64 bits; a warp holds such a row at one value per lane.
template <typename T, int VEC, int ITER, bool BLOCK, bool NEXT, typename S>
__global__ void __launch_bounds__(kMaxThreads) norm_bwd_kernel(const BwdParams p) {
  using P = Pack<T, VEC>;
  __shared__ float buf[2 * (kMaxThreads / 32) * kSums];
  int half = 0;
  const int nvec = p.d / VEC;
  const S inv_d = S(1) / (S)p.d;
  float acc_n[ITER][VEC], acc_p[ITER][VEC];
#pragma unroll
  for (int i = 0; i < ITER; ++i) {
#pragma unroll
    for (int c = 0; c < VEC; ++c) acc_n[i][c] = acc_p[i][c] = 0.0f;
  }
  for (int64_t row = blockIdx.x; row < p.T; row += gridDim.x) {
    const int64_t base = row * p.d;
    P pd[ITER], pn[ITER], po[ITER], py[ITER], pg[ITER];
#pragma unroll
    for (int i = 0; i < ITER; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      if (v >= nvec) continue;
      const int64_t at = base + (int64_t)v * VEC;
      if (p.dout) pd[i].load_once((const T *)p.dout + at);
      if (NEXT) {
        pn[i].load_once((const T *)p.dn + at);
        po[i].load_once((const T *)p.out + at);
      }
      if (BLOCK) {
        py[i].load_once((const T *)p.y + at);
        if (p.gate_kind == MOE_GATE_TOKEN) pg[i].load_once((const T *)p.gate + at);
        else if (p.gate_kind == MOE_GATE_CHANNEL) pg[i].load((const T *)p.gate + (int64_t)v * VEC);
      }
    }
    // out^2, out w_next dn | y^2, q dout, q w_next dn, q out
    S s[6] = {0, 0, 0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < ITER; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      if (v >= nvec) continue;
      float td[VEC], tn[VEC], to[VEC], ty[VEC], tw[VEC], tg[VEC];
      S u[VEC];
      P pw;
      if (NEXT) {
        pw.load((const T *)p.w_next + (int64_t)v * VEC);
        pw.unpack(tw);
        pn[i].unpack(tn);
        po[i].unpack(to);
#pragma unroll
        for (int c = 0; c < VEC; ++c) {
          u[c] = (S)tn[c] * tw[c];
          s[0] += (S)to[c] * to[c];
          s[1] += to[c] * u[c];
        }
      }
      if (BLOCK) {
        py[i].unpack(ty);
        pw.load((const T *)p.w_post + (int64_t)v * VEC);
        pw.unpack(tw);
        if (p.gate_kind != MOE_GATE_NONE) pg[i].unpack(tg);
        if (p.dout) pd[i].unpack(td);
#pragma unroll
        for (int c = 0; c < VEC; ++c) {
          s[2] += (S)ty[c] * ty[c];
          const S q = (S)ty[c] * tw[c] * (p.gate_kind != MOE_GATE_NONE ? tg[c] : 1.0f);
          if (p.dout) s[3] += q * td[c];
          if (NEXT) {
            s[4] += q * u[c];
            s[5] += q * to[c];
          }
        }
      }
    }
    block_sum(s, buf, half);
    const S rn = NEXT ? S(1) / sqrt(s[0] * inv_d + p.eps) : S(0);
    const S cn = rn * rn * (s[1] * inv_d);                   // r^2 mean(out u)
    const S ry = BLOCK ? S(1) / sqrt(s[2] * inv_d + p.eps) : S(0);
    const S uy = s[3] + rn * (s[4] - cn * s[5]);             // sum u y
    const S cy = ry * ry * (uy * inv_d);
#pragma unroll
    for (int i = 0; i < ITER; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      if (v >= nvec) continue;
      const int64_t at = base + (int64_t)v * VEC;
      float tn[VEC], to[VEC], ty[VEC], tw[VEC], tg[VEC], t[VEC];
      S G[VEC];
      P pw;
      if (p.dout) pd[i].unpack(t);
#pragma unroll
      for (int c = 0; c < VEC; ++c) G[c] = p.dout ? (S)t[c] : S(0);
      if (NEXT) {
        pw.load((const T *)p.w_next + (int64_t)v * VEC);
        pw.unpack(tw);
        pn[i].unpack(tn);
        po[i].unpack(to);
#pragma unroll
        for (int c = 0; c < VEC; ++c) {
          G[c] += rn * ((S)tn[c] * tw[c] - to[c] * cn);
          acc_n[i][c] = fmaf(tn[c] * (float)rn, to[c], acc_n[i][c]);
        }
      }
#pragma unroll
      for (int c = 0; c < VEC; ++c) t[c] = (float)(BLOCK ? p.res_scale * G[c] : G[c]);
      P::store((T *)p.dx + at, t);
      if (BLOCK) {
        py[i].unpack(ty);
        pw.load((const T *)p.w_post + (int64_t)v * VEC);
        pw.unpack(tw);
        if (p.gate_kind != MOE_GATE_NONE) pg[i].unpack(tg);
#pragma unroll
        for (int c = 0; c < VEC; ++c) {
          const float g = p.gate_kind != MOE_GATE_NONE ? tg[c] : 1.0f;
          const float Gy = (float)(G[c] * ty[c] * ry);
          acc_p[i][c] = p.gate_kind == MOE_GATE_TOKEN ? fmaf(g, Gy, acc_p[i][c]) : acc_p[i][c] + Gy;
          t[c] = (float)(ry * ((S)g * tw[c] * G[c] - ty[c] * cy));
          tg[c] = Gy * tw[c];
        }
        P::store((T *)p.dy + at, t);
        if (p.gate_kind == MOE_GATE_TOKEN) P::store((T *)p.d_gate + at, tg);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < ITER; ++i) {
    const int v = threadIdx.x + i * blockDim.x;
    if (v >= nvec) continue;
    float *dst = p.part + (int64_t)blockIdx.x * p.d + (int64_t)v * VEC;
#pragma unroll
    for (int c = 0; c < VEC; ++c) {
      if (NEXT) dst[c] = acc_n[i][c];
      if (BLOCK) dst[(int64_t)gridDim.x * p.d + c] = acc_p[i][c];
    }
  }
}

// Column sums of the blocks' partial rows, in a fixed order: 32 columns and 32 row groups per block.
template <typename T>
__global__ void __launch_bounds__(1024) norm_bwd_sum_kernel(const float *part, int blocks, int d, int gate_kind,
                                                            const T *w_post, const T *gate, T *dw_next, T *dw_post,
                                                            T *d_gate) {
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

// Vectors per row, per thread and threads per block for one row length: 16-byte vectors where a row is
// a multiple of 16 bytes, else single elements.
struct Shape {
  int vec, iter, threads;
};
static Shape shape_of(int d, int dtype) {
  const int full = dtype == MOE_BF16 ? 8 : 4;
  Shape s;
  s.vec = d % full == 0 ? full : 1;
  const int nvec = d / s.vec;
  s.iter = s.vec > 1 ? 1 : 4;
  while (s.iter * kMaxThreads < nvec) s.iter *= s.vec > 1 ? 2 : 4;
  const int per = (nvec + s.iter - 1) / s.iter;
  s.threads = (per + 31) / 32 * 32;
  return s;
}

// Blocks of the backward: each leaves a partial row, so there are no more than keep the GPU busy.
static int bwd_blocks(int64_t T, const Shape &s) {
  int64_t b = 152 * (s.threads >= 512 ? 2 : 1024 / s.threads);
  if (b > T) b = T;
  return b < 1 ? 1 : (int)b;
}

template <typename T, int VEC, int ITER>
static void launch_fwd(const FwdParams &p, bool block, bool next, int grid, int threads, cudaStream_t s) {
  if (!block) norm_fwd_kernel<T, VEC, ITER, false, true><<<grid, threads, 0, s>>>(p);
  else if (next) norm_fwd_kernel<T, VEC, ITER, true, true><<<grid, threads, 0, s>>>(p);
  else norm_fwd_kernel<T, VEC, ITER, true, false><<<grid, threads, 0, s>>>(p);
}
template <typename T, int VEC, int ITER, typename S = float>
static void launch_bwd(const BwdParams &p, bool block, bool next, int grid, int threads, cudaStream_t s) {
  if (!block) norm_bwd_kernel<T, VEC, ITER, false, true, S><<<grid, threads, 0, s>>>(p);
  else if (next) norm_bwd_kernel<T, VEC, ITER, true, true, S><<<grid, threads, 0, s>>>(p);
  else norm_bwd_kernel<T, VEC, ITER, true, false, S><<<grid, threads, 0, s>>>(p);
}

#define MOE_NORM_DISPATCH(FN, ...)                                        \
  do {                                                                    \
    if (dtype == MOE_BF16) {                                              \
      if (sh.vec == 8 && sh.iter == 1) FN<__nv_bfloat16, 8, 1>(__VA_ARGS__); \
      else if (sh.vec == 8) FN<__nv_bfloat16, 8, 2>(__VA_ARGS__);         \
      else if (sh.iter == 4) FN<__nv_bfloat16, 1, 4>(__VA_ARGS__);        \
      else FN<__nv_bfloat16, 1, 16>(__VA_ARGS__);                         \
    } else {                                                              \
      if (sh.vec == 4 && sh.iter == 1) FN<float, 4, 1>(__VA_ARGS__);      \
      else if (sh.vec == 4 && sh.iter == 2) FN<float, 4, 2>(__VA_ARGS__); \
      else if (sh.vec == 4) FN<float, 4, 4>(__VA_ARGS__);                 \
      else if (sh.iter == 4) FN<float, 1, 4>(__VA_ARGS__);                \
      else FN<float, 1, 16>(__VA_ARGS__);                                 \
    }                                                                     \
  } while (0)

static int check_shape(int T, int d, int dtype, float eps) {
  if (T < 0 || d < 1 || (dtype != MOE_F32 && dtype != MOE_BF16) || !(eps > 0.0f)) return MOE_ERR_INVALID_ARG;
  if (d > MOE_NORM_MAX_D) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}
static bool bad(const void *p) { return !p || !aligned16(p); }

static int run_fwd(const FwdParams &p, int dtype, bool block, bool next, cudaStream_t s) {
  const Shape sh = shape_of(p.d, dtype);
  int64_t grid = (int64_t)sm_count() * (2048 / sh.threads < 32 ? 2048 / sh.threads : 32);
  if (grid > p.T) grid = p.T;
  MOE_NORM_DISPATCH(launch_fwd, p, block, next, (int)grid, sh.threads, s);
  MOE_CHECK_LAUNCH();
  return MOE_OK;
}

static int run_bwd(BwdParams p, int dtype, bool block, bool next, void *dw_next, void *dw_post, void *d_gate, void *ws,
                   size_t ws_bytes, cudaStream_t s) {
  const Shape sh = shape_of(p.d, dtype);
  const int grid = bwd_blocks(p.T, sh);
  if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255) || ws_bytes < moe_norm_bwd_workspace_size((int)p.T, p.d, dtype))
    return MOE_ERR_INVALID_ARG;
  p.part = static_cast<float *>(ws);
  if (p.d <= 32) {
    if (dtype == MOE_BF16) launch_bwd<__nv_bfloat16, 1, 1, double>(p, block, next, grid, sh.threads, s);
    else launch_bwd<float, 1, 1, double>(p, block, next, grid, sh.threads, s);
  } else {
    MOE_NORM_DISPATCH(launch_bwd, p, block, next, grid, sh.threads, s);
  }
  MOE_CHECK_LAUNCH();
  const dim3 g((p.d + 31) / 32, block ? 2 : 1);
  if (dtype == MOE_BF16) {
    using B = __nv_bfloat16;
    norm_bwd_sum_kernel<B><<<g, 1024, 0, s>>>(p.part, grid, p.d, p.gate_kind, (const B *)p.w_post, (const B *)p.gate,
                                              (B *)dw_next, (B *)dw_post, (B *)d_gate);
  } else {
    norm_bwd_sum_kernel<float><<<g, 1024, 0, s>>>(p.part, grid, p.d, p.gate_kind, (const float *)p.w_post,
                                                  (const float *)p.gate, (float *)dw_next, (float *)dw_post,
                                                  (float *)d_gate);
  }
  MOE_CHECK_LAUNCH();
  return MOE_OK;
}

}  // namespace norm
}  // namespace moe

using namespace moe;
using namespace moe::norm;

extern "C" size_t moe_norm_bwd_workspace_size(int T, int d, int dtype) {
  if (T < 0 || d < 1) return 0;
  return (size_t)2 * bwd_blocks(T, shape_of(d, dtype)) * d * sizeof(float) + 256;
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
  if (bad(dw) || (T > 0 && (bad(dn) || bad(x) || bad(w) || bad(dx) || (dx_in && bad(dx_in))))) return MOE_ERR_INVALID_ARG;
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
