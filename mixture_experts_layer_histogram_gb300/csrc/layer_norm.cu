// Layer norm, forward and backward, and the norm that keeps its rows in 8 bits for the backward.
//
//   m = mean(x), r = 1 / sqrt(mean((x - m)^2) + eps), z = (x - m) r, n = z w + b
//   u = dn w,  dx = dx_in + r (u - mean(u) - z mean(u z)),  dw = sum_t dn z,  db = sum_t dn
//
// The forward leaves m and r (8 bytes a row) for the backward. m is the fp32 mean; what its rounding leaves,
// mean(x - m), is formed with the deviations and taken off again, in both directions, so a row far from zero loses nothing.
// Keeping: the forward also writes z as 8-bit codes with a power of two per 32 values (33 bytes per 32 values in the
// place of the 64 that x takes in bf16); restore() gives z w + b again for the block's own backward, and
// the backward reads z from the codes.
//
// HBM-bound, like the RMS norms (norm.cu): a thread block works on one row at a time, or on two, which share their reductions
// (the forward needs two per row, the deviations waiting for the mean), read once through the ring of rows and written once;
// codes come through the ring as well, 8 (fp32: 4) bytes per thread beside its 16-byte vectors. Rows whose length is no multiple
// of 16 bytes are read and written as the words that cover them (Windows), where there are enough of them. The weight gradients
// are summed over a block's rows in registers and its partial rows added up in a fixed order.
// Measured (bf16, in replayed graphs): T = 8192, d = 2048 forward 15.3 us (67 MB), with codes 19.7 (84 MB), restore 8.2 (51 MB),
// backward with dx_in 26 from x, 24.7 from codes (135 or 118 MB); T = 16384, d = 4096 forward 56, backward with dx_in 87 (537
// MB, 6.2 TB/s; 90 in a stream of calls with other inputs each time), from codes 85; d = 2047 forward 24.9, backward 48.7,
// keeping 8 bits 42.9, 15.0 and 58; fp32 T = 1023, d = 1537 forward 5.8, backward 8.8 us; four rows of 2048 2.3 and 4.0 us.
// Before dn and z stayed in registers between the backward's two passes it took 4% longer. Two vectors per thread or a warp per
// row (fewer instructions, no barriers) took the forward as long as one row at a time, 18.6 us.
#include <algorithm>
#include <type_traits>

#include "act8.cuh"
#include "raw16.cuh"
#include "row_ring.cuh"

namespace moe {
namespace norm {

// N sums over the block (N at most 4), the same on every thread: the exchanges of block_sum6, for four values.
template <int N> __device__ __forceinline__ void block_sums(float (&s)[N], SumBuf &buf, int &half) {
  const int lane = threadIdx.x & 31;
  float v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = i < N ? s[i < N ? i : 0] : 0.0f;
#pragma unroll
  for (int n = 2, off = 16; n >= 1; n >>= 1, off >>= 1) {
    const bool up = lane & off;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const float give = up ? v[i] : v[i + n], keep = up ? v[i + n] : v[i];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, give, off);
    }
  }
  float r = v[0];                                   // lanes 8 i .. 8 i + 7 carry value i
#pragma unroll
  for (int off = 4; off > 0; off >>= 1) r += __shfl_xor_sync(0xffffffffu, r, off);
  if (blockDim.x > 32) {
    float(*b)[kMaxWarps] = buf.v[half];
    half ^= 1;
    if ((lane & 7) == 0) b[lane >> 3][threadIdx.x >> 5] = r;
    __syncthreads();
    const float2 q = *reinterpret_cast<const float2 *>(&b[lane >> 3][2 * (lane & 7)]);
    r = q.x + q.y;
#pragma unroll
    for (int off = 4; off > 0; off >>= 1) r += __shfl_xor_sync(0xffffffffu, r, off);
  }
#pragma unroll
  for (int i = 0; i < N; ++i) s[i] = __shfl_sync(0xffffffffu, r, 8 * i);
}
template <int N> __device__ __forceinline__ void block_sums(double (&s)[N], SumBuf &, int &) {   // one warp
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
#pragma unroll
    for (int i = 0; i < N; ++i) s[i] += __shfl_xor_sync(0xffffffffu, s[i], off);
  }
}
static_assert(kMaxWarps == 16, "eight lanes read the warps' sums two at a time");

// Largest magnitude (fp32 bits) over a thread's VEC values and the other threads of its block of 32 values.
template <int VEC> __device__ __forceinline__ uint32_t block_amax(uint32_t m) {
#pragma unroll
  for (int off = 1; off < act8::kBlock / VEC; off <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, off));
  return m;
}
__device__ __forceinline__ float larger(float top, float v) { return act8::larger(top, v, 0.0f); }
__device__ __forceinline__ float larger(float top, F2 v) {
  float x, y;
  split(v, x, y);
  return act8::larger(top, x, y);
}
// The codes of N lanes of values times `inv`, written to p (VEC bytes)
__device__ __forceinline__ void put_codes(uint8_t *p, const F2 (&v)[4], float inv) {
  float f[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) split(mul(v[i], pair(inv, inv)), f[2 * i], f[2 * i + 1]);
  *reinterpret_cast<uint2 *>(p) = make_uint2(act8::pack4(f[0], f[1], f[2], f[3]), act8::pack4(f[4], f[5], f[6], f[7]));
}
__device__ __forceinline__ void put_codes(uint8_t *p, const F2 (&v)[2], float inv) {
  float f[4];
#pragma unroll
  for (int i = 0; i < 2; ++i) split(mul(v[i], pair(inv, inv)), f[2 * i], f[2 * i + 1]);
  *reinterpret_cast<uint32_t *>(p) = act8::pack4(f[0], f[1], f[2], f[3]);
}
__device__ __forceinline__ void put_codes(uint8_t *p, const float (&v)[1], float inv) { *p = act8::pack1(v[0] * inv); }
// The values of codes in shared memory (at their scale)
__device__ __forceinline__ void get_codes(uint32_t a, F2 (&v)[4], float scale) {
  uint32_t q[2];
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(q[0]), "=r"(q[1]) : "r"(a) : "memory");
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    float f[4];
    act8::unpack4(q[i], f);
    v[2 * i] = mul(pair(f[0], f[1]), pair(scale, scale));
    v[2 * i + 1] = mul(pair(f[2], f[3]), pair(scale, scale));
  }
}
__device__ __forceinline__ void get_codes(uint32_t a, F2 (&v)[2], float scale) {
  uint32_t q;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(q) : "r"(a) : "memory");
  float f[4];
  act8::unpack4(q, f);
  v[0] = mul(pair(f[0], f[1]), pair(scale, scale));
  v[1] = mul(pair(f[2], f[3]), pair(scale, scale));
}

// Rows that start anywhere, as vectors all the same: a block's rows lie so far apart (a multiple of 16 / sizeof(T) rows, or it
// has only one) that all of them start at the same place in a 16-byte word. Vectors are the words that cover a row, the ends of
// the first and the last one belong to other rows: their values count as zero, and are not written. Same use as Ring.
template <typename T, int VEC, int ITER> struct Windows {
  uint32_t mine, row_bytes, stage_bytes, step;
  int stages, d, nvec, lead;   // lead: values before the row in its first word
  int64_t all;                 // bytes of one tensor
  __device__ __forceinline__ Windows(const uint8_t *smem, const Geometry &g, int64_t rows, int d_)
      : row_bytes(g.row_bytes), stage_bytes(g.stage_bytes), stages(g.stages), d(d_) {
    lead = (int)((int64_t)blockIdx.x * d % VEC);
    nvec = (lead + d + VEC - 1) / VEC;
    mine = (uint32_t)__cvta_generic_to_shared(smem) + 16u * threadIdx.x;
    step = 16u * blockDim.x;
    all = rows * d * (int64_t)sizeof(T);
  }
  __device__ __forceinline__ bool has(int i) const { return (int)(threadIdx.x + i * blockDim.x) < nvec; }
  __device__ __forceinline__ int64_t offset(int64_t row) const { return (row * d - lead) * (int64_t)sizeof(T) + 16u * threadIdx.x; }
  // The column of the first value of this thread's i-th vector, and which of the vector's values are the row's
  __device__ __forceinline__ int column(int i) const { return (int)(threadIdx.x + i * blockDim.x) * VEC - lead; }
  __device__ __forceinline__ uint32_t valid(int i) const {
    uint32_t bits = 0;
#pragma unroll
    for (int c = 0; c < VEC; ++c) bits |= (uint32_t)((unsigned)(column(i) + c) < (unsigned)d) << c;
    return bits;
  }
  __device__ __forceinline__ void fetch(const void *base, int64_t off, int stage, int slot) const {
    const uint32_t dst = mine + (uint32_t)stage * stage_bytes + (uint32_t)slot * row_bytes;
    const uint8_t *src = (const uint8_t *)base + off;
#pragma unroll
    for (int i = 0; i < ITER; ++i) {
      if (!has(i)) continue;
      const int64_t left = all - off - i * step;   // up to the tensor's end: nothing past it is read
      const int n = left < 16 ? (int)left : 16;
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + i * step), "l"(src + i * step), "r"(n) : "memory");
    }
  }
  static __device__ __forceinline__ void commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
  __device__ __forceinline__ void wait() const {
    if (stages == 3) asm volatile("cp.async.wait_group 1;" ::: "memory");
    else asm volatile("cp.async.wait_group 0;" ::: "memory");
  }
  __device__ __forceinline__ uint32_t at(int stage, int64_t) const { return mine + (uint32_t)stage * stage_bytes; }
  __device__ __forceinline__ int freed(int stage) const { return stage >= 1 ? stage - 1 : stages - 1; }
};
template <int VEC> constexpr uint32_t kWhole = (1u << VEC) - 1;   // valid()
template <int N> __device__ __forceinline__ void only(F2 (&v)[N], uint32_t bits) {   // the values that are the row's, zeros for the others
#pragma unroll
  for (int c = 0; c < N; ++c) {
    float x, y;
    split(v[c], x, y);
    v[c] = pair(bits >> (2 * c) & 1 ? x : 0.0f, bits >> (2 * c + 1) & 1 ? y : 0.0f);
  }
}
template <typename T> __device__ __forceinline__ float value_at(const T *p) { return (float)*p; }
// A vector of w or b from any column on
template <typename T, int N> __device__ __forceinline__ void gather(const T *p, int column, uint32_t bits, F2 (&v)[N]) {
#pragma unroll
  for (int c = 0; c < N; ++c)
    v[c] = pair(bits >> (2 * c) & 1 ? value_at(p + column + 2 * c) : 0.0f, bits >> (2 * c + 1) & 1 ? value_at(p + column + 2 * c + 1) : 0.0f);
}
__device__ __forceinline__ void put_value(float *p, float v) { *p = v; }
__device__ __forceinline__ void put_value(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }
template <typename T, int N> __device__ __forceinline__ void scatter(T *p, uint32_t bits, const F2 (&v)[N]) {
#pragma unroll
  for (int c = 0; c < N; ++c) {
    float x, y;
    split(v[c], x, y);
    if (bits >> (2 * c) & 1) put_value(p + 2 * c, x);
    if (bits >> (2 * c + 1) & 1) put_value(p + 2 * c + 1, y);
  }
}
// A vector of a window lies in one block of 32 values or in two: `bound` of its values (those before the row's first counted)
// are the first one's.
struct Split {
  int b0, b1, bound;
  template <int VEC> static __device__ __forceinline__ Split of(int column, int d) {
    Split x;
    x.b0 = max(column, 0) / act8::kBlock;
    x.b1 = max(min(column + VEC, d) - 1, 0) / act8::kBlock;
    x.bound = min(max((x.b0 + 1) * act8::kBlock - column, 0), VEC);
    return x;
  }
};
// The values of a vector's codes, each at its block's scale
template <int N> __device__ __forceinline__ void at_scales(const uint32_t *q, float s0, float s1, int bound, F2 (&v)[N]) {
#pragma unroll
  for (int i = 0; i < N / 2; ++i) {
    float f[4];
    act8::unpack4(q[i], f);
#pragma unroll
    for (int c = 0; c < 4; ++c) f[c] *= 4 * i + c < bound ? s0 : s1;
    v[2 * i] = pair(f[0], f[1]);
    v[2 * i + 1] = pair(f[2], f[3]);
  }
}
template <int VEC> __device__ __forceinline__ void copy_codes(uint32_t dst, const uint8_t *src, int64_t left) {   // VEC of them, none past the end
  const int n = left < VEC ? (int)left : VEC;
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(VEC > 1 ? VEC : 4), "r"(n) : "memory");
}

template <typename T, int VEC, int ITER, bool WIN>
using RowsOf = typename std::conditional<WIN, Windows<T, VEC, ITER>, Ring<T, VEC, ITER>>::type;

struct LnFwdParams {
  const void *x, *w, *b;       // b may be null
  void *n;
  float *mean, *rstd;          // may be null
  uint8_t *codes, *scales;     // KEEP
  int64_t T;
  int d, nb;                   // nb: blocks of 32 per row
  float eps;
};

// rstd of a row from its mean m, what the rounding of m left, and the sum of the squared deviations from m; `write`: this thread
// writes the row's statistics.
__device__ __forceinline__ void statistics(const LnFwdParams &p, int64_t row, float m, float rest, float squares, float inv_d,
                                           bool write, float &r) {
  const float var = fmaf(-rest, rest, squares * inv_d);
  // squares past fp32's range: as if the variance were infinite
  r = squares == __uint_as_float(0x7f800000u) ? 0.0f : rsqrtf(fmaxf(var, 0.0f) + p.eps);
  if (var != var && squares != __uint_as_float(0x7f800000u)) r = var;   // (fmaxf drops a NaN)
  if (write) {
    if (p.mean) p.mean[row] = m + rest;
    if (p.rstd) p.rstd[row] = r;
  }
}
// Vector v of a row's normalised values to its codes (and, from the first thread of a block of 32 values, the scale)
template <int VEC, typename L, int N>
__device__ __forceinline__ void keep(const LnFwdParams &p, int64_t row, int v, bool has, const L (&z)[N]) {
  float top = 0.0f;
  if (has) {
#pragma unroll
    for (int c = 0; c < N; ++c) top = larger(top, z[c]);
  }
  const uint32_t byte = act8::scale_byte(block_amax<VEC>(__float_as_uint(top)));
  if (!has) return;
  uint8_t *q = p.codes + row * p.d + (int64_t)v * VEC;
  if (byte == 255u) {
#pragma unroll
    for (int c = 0; c < VEC; ++c) q[c] = 0;
  } else {
    put_codes(q, z, act8::inv_scale(byte));
  }
  if (v * VEC % act8::kBlock == 0) p.scales[row * p.nb + v * VEC / act8::kBlock] = (uint8_t)byte;
}

// keep() for a window's vector. The largest magnitudes of the row's blocks meet in shared memory (`tops`, fp32 bits, zeros at
// first) ...
template <int N> __device__ __forceinline__ void meet(uint32_t *tops, const Split &x, const F2 (&z)[N]) {
  float m0 = 0.0f, m1 = 0.0f;
#pragma unroll
  for (int c = 0; c < N; ++c) {
    float f[2];
    split(z[c], f[0], f[1]);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if (2 * c + k < x.bound) m0 = act8::larger(m0, f[k], 0.0f);
      else m1 = act8::larger(m1, f[k], 0.0f);
    }
  }
  atomicMax(tops + x.b0, __float_as_uint(m0));
  if (x.b1 != x.b0) atomicMax(tops + x.b1, __float_as_uint(m1));
}
// ... then codes, and the scales of the blocks that begin in this vector
template <int VEC, int N>
__device__ __forceinline__ void keep_window(const LnFwdParams &p, int64_t row, int column, uint32_t bits, const uint32_t *tops, const Split &x,
                                            const F2 (&z)[N]) {
  const uint32_t byte0 = act8::scale_byte(tops[x.b0]), byte1 = act8::scale_byte(tops[x.b1]);
  const float i0 = act8::inv_scale(byte0), i1 = act8::inv_scale(byte1);
  uint32_t w[N / 2];
#pragma unroll
  for (int i = 0; i < N / 2; ++i) {
    float f[4];
    split(z[2 * i], f[0], f[1]);
    split(z[2 * i + 1], f[2], f[3]);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const bool nan = (4 * i + c < x.bound ? byte0 : byte1) == 255u;
      f[c] = nan ? 0.0f : f[c] * (4 * i + c < x.bound ? i0 : i1);
    }
    w[i] = act8::pack4(f[0], f[1], f[2], f[3]);
  }
  uint8_t *q = p.codes + row * p.d + column;   // row * d - lead, and so this, is a multiple of VEC
  if (bits == kWhole<VEC>) {
    if constexpr (N == 4) *reinterpret_cast<uint2 *>(q) = make_uint2(w[0], w[1]);
    else *reinterpret_cast<uint32_t *>(q) = w[0];
  } else {
#pragma unroll
    for (int c = 0; c < VEC; ++c)
      if (bits >> c & 1) q[c] = (uint8_t)(w[c / 4] >> (8 * (c & 3)));
  }
  if (x.b0 * act8::kBlock >= column) p.scales[row * p.nb + x.b0] = (uint8_t)byte0;
  if (x.b1 != x.b0) p.scales[row * p.nb + x.b1] = (uint8_t)byte1;
}

// ROWS: rows that a block takes at a time, which share the reductions' exchanges and barriers. WIN: Windows.
template <typename T, int VEC, int ITER, bool KEEP, int ROWS, bool WIN>
__global__ void __launch_bounds__(kMaxThreads, ITER == 1 ? 2 : 1) ln_fwd_kernel(const LnFwdParams p, const Geometry geom) {
  using V = Lanes<T, VEC, float>;
  using L = typename V::L;
  constexpr int N = V::N;
  constexpr bool kHold = ITER * VEC <= 16 && ITER <= 4;
  static_assert(!WIN || kHold, "windows hold their weights");
  extern __shared__ __align__(16) uint8_t dyn[];
  __shared__ SumBuf sums;
  __shared__ uint32_t tops[WIN && KEEP ? 2 : 1][ROWS][WIN && KEEP ? MOE_NORM_MAX_D / act8::kBlock : 1];   // two turns' in turn
  int tops_at = 0;
  const RowsOf<T, VEC, ITER, WIN> ring(dyn, geom, p.T, p.d);
  uint32_t bits[WIN ? ITER : 1];
  if constexpr (WIN) {
#pragma unroll
    for (int i = 0; i < ITER; ++i) bits[i] = ring.valid(i);
  }
  int half = 0;
  const float inv_d = 1.0f / (float)p.d;
  clear(sums);
  // The rows of one turn lie gridDim.x apart.
  const int64_t turn = (int64_t)ROWS * gridDim.x;
  auto fetch = [&](int64_t row, int stage) {
#pragma unroll
    for (int j = 0; j < ROWS; ++j, row += gridDim.x)
      if (row < p.T) ring.fetch(p.x, ring.offset(row), stage, j);
    ring.commit();
  };
  for (int s = 0; s < ring.stages - 1; ++s) fetch(blockIdx.x + s * turn, s);
  auto weights = [&](int v, L *w, L *b) {
    V::load((const T *)p.w + (int64_t)v * VEC, w);
    if (p.b) {
      V::load((const T *)p.b + (int64_t)v * VEC, b);
    } else {
#pragma unroll
      for (int c = 0; c < N; ++c) b[c] = splat<L>(0.0f);
    }
  };
  L hold_w[kHold ? ITER : 1][N], hold_b[kHold ? ITER : 1][N];
  if constexpr (WIN) {
#pragma unroll
    for (int i = 0; i < ITER; ++i) {
      gather((const T *)p.w, ring.column(i), bits[i], hold_w[i]);
      gather((const T *)p.b, ring.column(i), p.b ? bits[i] : 0, hold_b[i]);
    }
  } else if (kHold) {
#pragma unroll
    for (int i = 0; i < ITER; ++i)
      if (ring.has(i)) weights(threadIdx.x + i * blockDim.x, hold_w[kHold ? i : 0], hold_b[kHold ? i : 0]);
  }
  int stage = 0;
  for (int64_t row = blockIdx.x; row < p.T; row += turn) {
    if (ring.stages == 1) {
      if (VEC == 1) __syncthreads();   // every thread has left the rows before
      fetch(row, 0);
    }
    ring.wait();
    if constexpr (WIN && KEEP) {   // (read last two turns ago; the sums' barriers come before this turn's writes)
      for (int i = threadIdx.x; i < ROWS * p.nb; i += blockDim.x) tops[tops_at][i / p.nb][i % p.nb] = 0;
      if (blockDim.x == 32) __syncwarp();
    }
    L o[ROWS][ITER][N];
    float m[ROWS];
#pragma unroll
    for (int j = 0; j < ROWS; ++j) {
      L s = splat<L>(0.0f);
      if (j == 0 || row + j * gridDim.x < p.T) {
        const uint32_t here = ring.at(stage, ring.offset(row + j * gridDim.x)) + j * ring.row_bytes;
#pragma unroll
        for (int i = 0; i < ITER; ++i) {
          if (!ring.has(i)) continue;
          V::load_shared(here + i * ring.step, o[j][i]);
          if constexpr (WIN) {
            if (bits[i] != kWhole<VEC>) only(o[j][i], bits[i]);
          }
#pragma unroll
          for (int c = 0; c < N; ++c) s = add(s, o[j][i][c]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < ITER; ++i) {
#pragma unroll
          for (int c = 0; c < N; ++c) o[j][i][c] = splat<L>(0.0f);
        }
      }
      m[j] = total(s);
    }
    // the rows are in registers: the stage of those before them may be overwritten
    if (ring.stages > 1) fetch(row + (ring.stages - 1) * turn, ring.freed(stage));
    if constexpr (ROWS == 1) m[0] = block_sum(m[0], sums, half);
    else block_sums(m, sums, half);
    float t[2 * ROWS];   // sums of the deviations (what the rounding of m left), and of their squares
#pragma unroll
    for (int j = 0; j < ROWS; ++j) {
      m[j] *= inv_d;
      L s1 = splat<L>(0.0f), s2 = splat<L>(0.0f);
      const L minus = splat<L>(-m[j]);
#pragma unroll
      for (int i = 0; i < ITER; ++i) {
        if (!ring.has(i)) continue;
#pragma unroll
        for (int c = 0; c < N; ++c) o[j][i][c] = add(o[j][i][c], minus);
        if constexpr (WIN) {
          if (bits[i] != kWhole<VEC>) only(o[j][i], bits[i]);
        }
#pragma unroll
        for (int c = 0; c < N; ++c) {
          s1 = add(s1, o[j][i][c]);
          s2 = fma(o[j][i][c], o[j][i][c], s2);
        }
      }
      t[2 * j] = total(s1);
      t[2 * j + 1] = total(s2);
    }
    block_sums(t, sums, half);
#pragma unroll
    for (int j = 0; j < ROWS; ++j) {
      const int64_t r_ = row + j * gridDim.x;
      if (j > 0 && r_ >= p.T) break;
      const float rest = t[2 * j] * inv_d;
      float r;
      statistics(p, r_, m[j], rest, t[2 * j + 1], inv_d, threadIdx.x == 0, r);
      const L R = splat<L>(r), shift = splat<L>(-rest * r);
#pragma unroll
      for (int i = 0; i < ITER; ++i) {
        if (!ring.has(i)) continue;
#pragma unroll
        for (int c = 0; c < N; ++c) o[j][i][c] = fma(o[j][i][c], R, shift);
        if constexpr (WIN && KEEP) {
          if (bits[i] != kWhole<VEC>) only(o[j][i], bits[i]);
          meet(tops[tops_at][j], Split::of<VEC>(ring.column(i), p.d), o[j][i]);
        }
      }
    }
    if constexpr (WIN && KEEP) __syncthreads();
#pragma unroll
    for (int j = 0; j < ROWS; ++j) {
      const int64_t r_ = row + j * gridDim.x;
      if (j > 0 && r_ >= p.T) break;
#pragma unroll
      for (int i = 0; i < ITER; ++i) {
        const int v = threadIdx.x + i * blockDim.x;
        if constexpr (KEEP && !WIN) keep<VEC>(p, r_, v, ring.has(i), o[j][i]);
        if (!ring.has(i)) continue;
        if constexpr (KEEP && WIN)
          keep_window<VEC>(p, r_, ring.column(i), bits[i], tops[tops_at][j], Split::of<VEC>(ring.column(i), p.d), o[j][i]);
        L(&w)[N] = hold_w[kHold ? i : 0], (&b)[N] = hold_b[kHold ? i : 0];
        if (!kHold) weights(v, w, b);
#pragma unroll
        for (int c = 0; c < N; ++c) o[j][i][c] = fma(o[j][i][c], w[c], b[c]);
        T *out = reinterpret_cast<T *>((uint8_t *)p.n + ring.offset(r_) + (VEC > 1 ? 0u : (uint32_t)sizeof(T) * threadIdx.x) + i * ring.step);
        if constexpr (WIN) {
          if (bits[i] != kWhole<VEC>) {
            scatter(out, bits[i], o[j][i]);
            continue;
          }
        }
        V::store(out, o[j][i]);
      }
    }
    tops_at ^= 1;
    if (++stage == ring.stages) stage = 0;
  }
}

struct LnBwdParams {
  const void *dn, *x, *dx_in, *w;     // dx_in may be null; x unless KEPT
  const float *mean, *rstd;           // mean unless KEPT
  const uint8_t *codes, *scales;      // KEPT
  void *dx;
  float *part;                        // [2][blocks][d]: dw, then db
  int64_t T;
  int d, nb;
  float eps;
};

// S: float, or double for rows of at most 32 values, where u - mean(u) - z mean(u z) all but cancels (in a row of one or two
// values what is left is of the order of eps): such rows are computed in 64 bits from x itself, its statistics too.
// ROWS, WIN: as in the forward.
template <typename T, int VEC, int ITER, bool KEPT, typename S, int ROWS, bool WIN>
__global__ void __launch_bounds__(kMaxThreads, VEC == 1 && ITER <= 4 ? 2 : 1) ln_bwd_kernel(const LnBwdParams p, const Geometry geom) {
  using V = Lanes<T, VEC, S>;
  using L = typename V::L;
  constexpr int N = V::N;
  constexpr bool kWide = sizeof(S) == 8;
  constexpr bool kHold = ITER * VEC <= 16 && ITER <= 4;
  static_assert(ROWS == 1 || (VEC > 1 && kHold), "several rows at a time stay in registers");
  static_assert(!WIN || kHold, "windows hold their weights");
  constexpr int kDn = 0, kX = 1, kIn = 2;    // a row's buffers in a stage; kX holds the codes where they are copied
  extern __shared__ __align__(16) uint8_t dyn[];
  __shared__ SumBuf sums;
  const RowsOf<T, VEC, ITER, WIN> ring(dyn, geom, p.T, p.d);
  uint32_t bits[WIN ? ITER : 1];
  if constexpr (WIN) {
#pragma unroll
    for (int i = 0; i < ITER; ++i) bits[i] = ring.valid(i);
  }
  int half = 0;
  const S inv_d = S(1) / (S)p.d;
  const bool has_in = p.dx_in != nullptr;
  const int per_row = has_in ? 3 : 2;
  const uint32_t codes_at = VEC > 1 ? (uint32_t)kX * ring.row_bytes - (16u - VEC) * threadIdx.x : 0u;   // from ring.mine
  clear(sums);
  const int64_t turn = (int64_t)ROWS * gridDim.x;   // the rows of one turn lie gridDim.x apart
  auto fetch = [&](int64_t row, int stage) {
#pragma unroll
    for (int j = 0; j < ROWS; ++j, row += gridDim.x) {
      if (row >= p.T) break;
      const int64_t off = ring.offset(row);
      const int at = j * per_row;
      ring.fetch(p.dn, off, stage, at + kDn);
      if (!KEPT) {
        ring.fetch(p.x, off, stage, at + kX);
      } else if (VEC > 1) {   // VEC bytes per vector, copied by the thread that reads them
        const uint32_t dst = ring.mine + (uint32_t)stage * ring.stage_bytes + codes_at + at * ring.row_bytes;
        const int64_t first = row * p.d + VEC * threadIdx.x;
#pragma unroll
        for (int i = 0; i < ITER; ++i) {
          if (!ring.has(i)) continue;
          const int64_t from = first + i * VEC * blockDim.x;
          if constexpr (WIN) copy_codes<VEC>(dst + i * VEC * blockDim.x, p.codes + from - ring.lead, p.T * p.d - from + ring.lead);
          else copy_codes<VEC>(dst + i * VEC * blockDim.x, p.codes + from, VEC);
        }
      }
      if (has_in) ring.fetch(p.dx_in, off, stage, at + kIn);
    }
    ring.commit();
  };
  L acc_w[ITER][N], acc_b[ITER][N];
#pragma unroll
  for (int i = 0; i < ITER; ++i) {
#pragma unroll
    for (int c = 0; c < N; ++c) acc_w[i][c] = acc_b[i][c] = splat<L>(0.0f);
  }
  for (int s = 0; s < ring.stages - 1; ++s) fetch(blockIdx.x + s * turn, s);
  L hold_w[kHold ? ITER : 1][N];
  if constexpr (WIN) {
#pragma unroll
    for (int i = 0; i < ITER; ++i) gather((const T *)p.w, ring.column(i), bits[i], hold_w[i]);
  } else if (kHold) {
#pragma unroll
    for (int i = 0; i < ITER; ++i)
      if (ring.has(i)) V::load((const T *)p.w + (int64_t)(threadIdx.x + i * blockDim.x) * VEC, hold_w[kHold ? i : 0]);
  }
  // the rows' statistics, and the scales of this thread's codes, are read one turn ahead
  float next_m[ROWS] = {}, next_r[ROWS] = {};
  uint8_t next_s[ROWS][KEPT ? ITER : 1] = {}, next_s1[ROWS][KEPT && WIN ? ITER : 1] = {};   // next_s1: of the second block
  auto ahead = [&](int64_t row) {
#pragma unroll
    for (int j = 0; j < ROWS; ++j, row += gridDim.x) {
      if (row >= p.T) break;
      if (!KEPT) next_m[j] = p.mean[row];
      next_r[j] = p.rstd[row];
      if (KEPT) {
#pragma unroll
        for (int i = 0; i < ITER; ++i) {
          if (!ring.has(i)) continue;
          if constexpr (WIN) {
            const Split x = Split::of<VEC>(ring.column(i), p.d);
            next_s[j][KEPT ? i : 0] = p.scales[row * p.nb + x.b0];
            next_s1[j][KEPT && WIN ? i : 0] = p.scales[row * p.nb + x.b1];
          } else {
            next_s[j][KEPT ? i : 0] = p.scales[row * p.nb + (int)(threadIdx.x + i * blockDim.x) * VEC / act8::kBlock];
          }
        }
      }
    }
  };
  ahead(blockIdx.x);
  int stage = 0;
  for (int64_t row = blockIdx.x; row < p.T; row += turn) {
    if (ring.stages == 1) {
      if (VEC == 1) __syncthreads();   // every thread has left the rows before
      fetch(row, 0);
    }
    S m[ROWS], r[ROWS];
    float sc[ROWS][KEPT ? ITER : 1], sc1[ROWS][KEPT && WIN ? ITER : 1];
#pragma unroll
    for (int j = 0; j < ROWS; ++j) {
      m[j] = next_m[j];
      r[j] = next_r[j];
      if (KEPT) {
#pragma unroll
        for (int i = 0; i < ITER; ++i) {
          sc[j][KEPT ? i : 0] = act8::scale_value(next_s[j][KEPT ? i : 0]);
          if (WIN) sc1[j][KEPT && WIN ? i : 0] = act8::scale_value(next_s1[j][KEPT && WIN ? i : 0]);
        }
      }
    }
    ahead(row + turn);
    ring.wait();
    // every thread has left the rows before (words: it reads what it has copied itself; single values: the barrier in wait())
    if (ring.stages > 1) fetch(row + (ring.stages - 1) * turn, ring.freed(stage));
    const int64_t off0 = ring.offset(row);
    const uint32_t here = ring.at(stage, off0);
    const uint32_t codes_here = ring.mine + (uint32_t)stage * ring.stage_bytes + codes_at;
    if constexpr (kWide && !KEPT) {   // one value per lane
      S t[1] = {S(0)};
      L x[N];
      x[0] = S(0);
      if (ring.has(0)) V::load_shared(here + kX * ring.row_bytes, x);
      t[0] = x[0];
      block_sums(t, sums, half);
      m[0] = t[0] * inv_d;
      t[0] = ring.has(0) ? (x[0] - m[0]) * (x[0] - m[0]) : S(0);
      block_sums(t, sums, half);
      // a stored 0: squares past fp32's range, whose row the forward took for one of infinite variance (z = 0)
      if (r[0] != S(0)) r[0] = S(1) / sqrt(t[0] * inv_d + (S)p.eps);
    }
    // z (without KEPT: before the rest of the mean is taken off) of the i-th vector of the j-th row
    auto normed = [&](int j, int i, L (&z)[N]) {
      if constexpr (KEPT) {
        if constexpr (WIN) {
          uint32_t q[N / 2];
          const uint32_t a = codes_here + j * per_row * ring.row_bytes + i * VEC * blockDim.x;
#pragma unroll
          for (int k = 0; k < N / 2; ++k) asm volatile("ld.shared.u32 %0, [%1];" : "=r"(q[k]) : "r"(a + 4 * k) : "memory");
          at_scales(q, sc[j][i], sc1[j][i], Split::of<VEC>(ring.column(i), p.d).bound, z);
        } else if constexpr (VEC > 1) {
          get_codes(codes_here + j * per_row * ring.row_bytes + i * VEC * blockDim.x, z, sc[j][i]);
        } else {
          z[0] = (S)(act8::unpack1(p.codes[row * p.d + threadIdx.x + (int64_t)i * blockDim.x]) * sc[j][i]);
        }
      } else {
        V::load_shared(here + (j * per_row + kX) * ring.row_bytes + i * ring.step, z);
#pragma unroll
        for (int c = 0; c < N; ++c) z[c] = mul(add(z[c], all(-m[j], L())), all(r[j], L()));
      }
    };
    // sums of u, u z, z; with few vectors per thread dn and z stay in registers for the second pass
    constexpr int SUMS = KEPT ? 2 : 3;
    L hold_d[ROWS][kHold ? ITER : 1][N], hold_z[ROWS][kHold ? ITER : 1][N];
    S s[SUMS * ROWS];
#pragma unroll
    for (int j = 0; j < ROWS; ++j) {
      L t[3];
#pragma unroll
      for (int i = 0; i < 3; ++i) t[i] = splat<L>(0.0f);
      if (j == 0 || row + j * gridDim.x < p.T) {
#pragma unroll
        for (int i = 0; i < ITER; ++i) {
          if (!ring.has(i)) continue;
          L(&w)[N] = hold_w[kHold ? i : 0];
          if (!kHold) V::load((const T *)p.w + (int64_t)(threadIdx.x + i * blockDim.x) * VEC, w);
          L(&u)[N] = hold_d[j][kHold ? i : 0], (&z)[N] = hold_z[j][kHold ? i : 0];
          V::load_shared(here + (j * per_row + kDn) * ring.row_bytes + i * ring.step, u);
          normed(j, i, z);
          if constexpr (WIN) {
            if (bits[i] != kWhole<VEC>) {
              only(u, bits[i]);
              only(z, bits[i]);
            }
          }
#pragma unroll
          for (int c = 0; c < N; ++c) {
            acc_b[i][c] = add(acc_b[i][c], u[c]);
            const L uw = mul(u[c], w[c]);
            t[0] = add(t[0], uw);
            t[1] = fma(uw, z[c], t[1]);
            if (!KEPT) t[2] = add(t[2], z[c]);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < SUMS; ++i) s[SUMS * j + i] = total(t[i]);
    }
    if constexpr (SUMS * ROWS == 6) block_sum6(s, sums, half);
    else block_sums(s, sums, half);
#pragma unroll
    for (int j = 0; j < ROWS; ++j) {
      if (j > 0 && row + j * gridDim.x >= p.T) break;
      const int64_t off = j == 0 ? off0 : ring.offset(row + j * gridDim.x);
      const S rest = KEPT ? S(0) : s[SUMS * j + SUMS - 1] * inv_d;   // of z's mean, which is zero
      const S mu = s[SUMS * j] * inv_d, muz = (s[SUMS * j + 1] - rest * s[SUMS * j]) * inv_d;
      const L R = all(r[j], L()), Rest = all(-rest, L()), Mu = all(-mu, L()), Muz = all(-muz, L());
#pragma unroll
      for (int i = 0; i < ITER; ++i) {
        if (!ring.has(i)) continue;
        L(&w)[N] = hold_w[kHold ? i : 0];
        if (!kHold) V::load((const T *)p.w + (int64_t)(threadIdx.x + i * blockDim.x) * VEC, w);
        L(&u)[N] = hold_d[j][kHold ? i : 0], (&z)[N] = hold_z[j][kHold ? i : 0];
        L g[N];
        if (!kHold) {
          V::load_shared(here + kDn * ring.row_bytes + i * ring.step, u);
          normed(j, i, z);
        }
        if (has_in) {
          V::load_shared(here + (j * per_row + kIn) * ring.row_bytes + i * ring.step, g);
        } else {
#pragma unroll
          for (int c = 0; c < N; ++c) g[c] = splat<L>(0.0f);
        }
#pragma unroll
        for (int c = 0; c < N; ++c) {
          if (!KEPT) z[c] = add(z[c], Rest);
          acc_w[i][c] = fma(u[c], z[c], acc_w[i][c]);
          g[c] = fma(fma(z[c], Muz, fma(u[c], w[c], Mu)), R, g[c]);
        }
        T *out = reinterpret_cast<T *>((uint8_t *)p.dx + off + (VEC > 1 ? 0u : (uint32_t)sizeof(T) * threadIdx.x) + i * ring.step);
        if constexpr (WIN) {
          if (bits[i] != kWhole<VEC>) {
            scatter(out, bits[i], g);
            continue;
          }
        }
        V::store(out, g);
      }
    }
    if (++stage == ring.stages) stage = 0;
  }
  start_next();   // the kernel that adds up the partial rows
#pragma unroll
  for (int i = 0; i < ITER; ++i) {
    if (!ring.has(i)) continue;
    if constexpr (WIN) {
      float *dst = p.part + (int64_t)blockIdx.x * p.d + ring.column(i);
      scatter(dst, bits[i], acc_w[i]);
      scatter(dst + (int64_t)gridDim.x * p.d, bits[i], acc_b[i]);
    } else {
      float *dst = p.part + (int64_t)blockIdx.x * p.d + (int64_t)(threadIdx.x + i * blockDim.x) * VEC;
      put_part(dst, acc_w[i]);
      put_part(dst + (int64_t)gridDim.x * p.d, acc_b[i]);
    }
  }
}

// n = z w + b of kept rows. A thread keeps its columns (VEC of them) and takes every `step`-th row.
constexpr int kRestoreThreads = 256;
// 16 values of bf16 rows of whole blocks: 16-byte loads, 32-byte stores
__global__ void __launch_bounds__(kRestoreThreads) ln_restore16_kernel(const uint4 *__restrict__ codes,
                                                                       const uint8_t *__restrict__ scales,
                                                                       const __nv_bfloat16 *__restrict__ w,
                                                                       const __nv_bfloat16 *__restrict__ b, int64_t T_, int d,
                                                                       int64_t step, bool wide, __nv_bfloat16 *__restrict__ n) {
  const int cols = d / 16;
  const int64_t id = (int64_t)blockIdx.x * kRestoreThreads + threadIdx.x;
  const int64_t row0 = id / cols;
  const int col = (int)(id - row0 * cols);
  if (row0 >= step) return;
  Raw16<__nv_bfloat16> raw;
  float W[16], B[16] = {};
  raw.load(w + col * 16);
  raw.unpack(W);
  if (b) {
    raw.load(b + col * 16);
    raw.unpack(B);
  }
  constexpr int kRows = 4;   // in flight
  for (int64_t r0 = row0; r0 < T_; r0 += kRows * step) {
    uint4 q[kRows];
    uint32_t sc[kRows];
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
      const int64_t at = (r0 + k * step) * cols + col;
      if (r0 + k * step >= T_) continue;
      q[k] = __ldg(codes + at);
      sc[k] = __ldg(scales + (at >> 1));
    }
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
      if (r0 + k * step >= T_) continue;
      const float scale = act8::scale_value(sc[k]);
      float v[16];
      act8::unpack4(q[k].x, v);
      act8::unpack4(q[k].y, v + 4);
      act8::unpack4(q[k].z, v + 8);
      act8::unpack4(q[k].w, v + 12);
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = fmaf(v[i] * scale, W[i], B[i]);
      Raw16<__nv_bfloat16>::store(n + (r0 + k * step) * d + col * 16, v, wide);
    }
  }
}

template <typename T, int VEC>
__global__ void __launch_bounds__(kRestoreThreads) ln_restore_kernel(const uint8_t *__restrict__ codes,
                                                                     const uint8_t *__restrict__ scales,
                                                                     const T *__restrict__ w, const T *__restrict__ b, int64_t T_,
                                                                     int d, int nb, int64_t step, T *__restrict__ n) {
  using V = Lanes<T, VEC, float>;
  using L = typename V::L;
  constexpr int N = V::N;
  const int cols = d / VEC;
  const int64_t id = (int64_t)blockIdx.x * kRestoreThreads + threadIdx.x;
  const int64_t row0 = id / cols;
  const int col = (int)(id - row0 * cols) * VEC;
  if (row0 >= step) return;
  L W[N], B[N];
  V::load(w + col, W);
  if (b) {
    V::load(b + col, B);
  } else {
#pragma unroll
    for (int c = 0; c < N; ++c) B[c] = splat<L>(0.0f);
  }
  constexpr int kRows = 4;   // in flight
  for (int64_t r0 = row0; r0 < T_; r0 += kRows * step) {
    uint32_t q[kRows][VEC >= 4 ? VEC / 4 : 1];
    float sc[kRows];
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
      const int64_t r = r0 + k * step;
      if (r >= T_) continue;
      const uint8_t *src = codes + r * d + col;
      if constexpr (VEC == 8) {
        const uint2 v = __ldg(reinterpret_cast<const uint2 *>(src));
        q[k][0] = v.x;
        q[k][VEC >= 8 ? 1 : 0] = v.y;
      } else if constexpr (VEC == 4) {
        q[k][0] = __ldg(reinterpret_cast<const uint32_t *>(src));
      } else {
        q[k][0] = __ldg(src);
      }
      sc[k] = act8::scale_value(__ldg(scales + r * nb + col / act8::kBlock));
    }
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
      const int64_t r = r0 + k * step;
      if (r >= T_) continue;
      L v[N];
      if constexpr (VEC == 1) {
        v[0] = act8::unpack1((uint8_t)q[k][0]) * sc[k];
      } else {
#pragma unroll
        for (int i = 0; i < VEC / 4; ++i) {
          float f[4];
          act8::unpack4(q[k][i], f);
          v[2 * i] = mul(pair(f[0], f[1]), pair(sc[k], sc[k]));
          v[2 * i + 1] = mul(pair(f[2], f[3]), pair(sc[k], sc[k]));
        }
      }
#pragma unroll
      for (int c = 0; c < N; ++c) v[c] = fma(v[c], W[c], B[c]);
      V::store(n + r * d + col, v);
    }
  }
}

// Rows that start anywhere: a thread's rows lie a multiple of VEC apart, so its words start at the same column in all of them.
template <typename T, int VEC>
__global__ void __launch_bounds__(kRestoreThreads) ln_restore_windows_kernel(const uint8_t *__restrict__ codes,
                                                                             const uint8_t *__restrict__ scales,
                                                                             const T *__restrict__ w, const T *__restrict__ b,
                                                                             int64_t T_, int d, int nb, int words, int64_t step,
                                                                             T *__restrict__ n) {
  using V = Lanes<T, VEC, float>;
  constexpr int N = V::N;
  const int64_t id = (int64_t)blockIdx.x * kRestoreThreads + threadIdx.x, row0 = id / words;
  if (row0 >= step) return;
  const int column = (int)(id - row0 * words) * VEC - (int)(row0 * d % VEC);
  uint32_t bits = 0;
#pragma unroll
  for (int c = 0; c < VEC; ++c) bits |= (uint32_t)((unsigned)(column + c) < (unsigned)d) << c;
  if (bits == 0) return;
  F2 W[N], B[N];
  gather(w, column, bits, W);
  gather(b, column, b ? bits : 0, B);
  const Split x = Split::of<VEC>(column, d);
  constexpr int kRows = 4;   // in flight
  for (int64_t r0 = row0; r0 < T_; r0 += kRows * step) {
    uint32_t q[kRows][N / 2];
    float s0[kRows], s1[kRows];
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
      const int64_t r = r0 + k * step;
      if (r >= T_) continue;
      const uint8_t *src = codes + r * d + column;
      if (bits == kWhole<VEC>) {
        if constexpr (N == 4) {
          const uint2 v = __ldg(reinterpret_cast<const uint2 *>(src));
          q[k][0] = v.x;
          q[k][N / 2 - 1] = v.y;
        } else {
          q[k][0] = __ldg(reinterpret_cast<const uint32_t *>(src));
        }
      } else {
#pragma unroll
        for (int i = 0; i < N / 2; ++i) q[k][i] = 0;
#pragma unroll
        for (int c = 0; c < VEC; ++c)
          if (bits >> c & 1) q[k][c / 4] |= (uint32_t)__ldg(src + c) << (8 * (c & 3));
      }
      s0[k] = act8::scale_value(__ldg(scales + r * nb + x.b0));
      s1[k] = act8::scale_value(__ldg(scales + r * nb + x.b1));
    }
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
      const int64_t r = r0 + k * step;
      if (r >= T_) continue;
      F2 v[N];
      at_scales(q[k], s0[k], s1[k], x.bound, v);
#pragma unroll
      for (int c = 0; c < N; ++c) v[c] = fma(v[c], W[c], B[c]);
      T *out = n + r * d + column;
      if (bits == kWhole<VEC>) V::store(out, v);
      else scatter(out, bits, v);
    }
  }
}

// Rows of words for rows that start anywhere; vec 1 where a thread would have to hold too many values (bf16 from 8186 values on, fp32
// from 8190).
static Shape windows_of(int d, int dtype) {
  const int es = dtype == MOE_BF16 ? 2 : 4, vec = 16 / es, nvec = (d + 2 * vec - 2) / vec;   // words, wherever the row starts
  Shape s;
  s.vec = vec;
  // Two words per thread where a block of more than 256 threads would have an SM to itself: always for fp32 (35 against 43 us
  // for the backward at 8192 x 1537), for bf16 while it would be few more (49 against 52 at 8192 x 2047; 67 against 57 at 8192 x
  // 3001).
  s.iter = nvec > kMaxThreads / 2 && (dtype == MOE_F32 || nvec <= 320) ? 2 : 1;
  while (s.iter * kMaxThreads < nvec) s.iter *= 2;
  s.threads = ((nvec + s.iter - 1) / s.iter + 31) / 32 * 32;
  s.row_bytes = (uint32_t)nvec * 16;
  if (s.iter * vec > 16) s.vec = 1;
  return s;
}

template <typename T, int VEC, int ITER, bool WIN> static int ln_launch_fwd(const LnFwdParams &p, const Shape &sh, cudaStream_t s) {
  const int threads = sh.iter == 1 ? 2 * kMaxThreads : kMaxThreads;
  const int64_t sms = sm_count() / 8 * 8;   // (of windows all rows of a block have to start alike)
  int64_t grid = sms * per_sm(sh, 1, threads);
  // Two rows at a time where a thread has one vector of each and blocks have more rows than one: 16.4 against 18.6 us at T =
  // 8192, d = 2048 bf16, 58.6 against 71.9 at 16384 x 4096; for four rows 2.5 against 2.3 (nothing is shared then).
  if constexpr (VEC > 1 && ITER == 1) {
    if (p.T > grid) {
      grid = sms * per_sm(sh, 2, threads);
      if (grid > p.T) grid = p.T;
      if (p.codes) return launch<ln_fwd_kernel<T, VEC, ITER, true, 2, WIN>>(p, sh, 2, (int)grid, s);
      return launch<ln_fwd_kernel<T, VEC, ITER, false, 2, WIN>>(p, sh, 2, (int)grid, s);
    }
  }
  if (grid > p.T) grid = p.T;
  if (p.codes) return launch<ln_fwd_kernel<T, VEC, ITER, true, 1, WIN>>(p, sh, 1, (int)grid, s);
  return launch<ln_fwd_kernel<T, VEC, ITER, false, 1, WIN>>(p, sh, 1, (int)grid, s);
}
template <typename T, int VEC, int ITER, bool WIN, typename S = float>
static int ln_launch_bwd(const LnBwdParams &p, const Shape &sh, int rows, int grid, cudaStream_t s) {
  const int tensors = rows * (p.dx_in ? 3 : 2);
  if constexpr (VEC > 1 && ITER == 1) {
    if (rows == 2) {
      if (p.codes) return launch<ln_bwd_kernel<T, VEC, ITER, true, S, 2, WIN>>(p, sh, tensors, grid, s);
      return launch<ln_bwd_kernel<T, VEC, ITER, false, S, 2, WIN>>(p, sh, tensors, grid, s);
    }
  }
  if (p.codes) return launch<ln_bwd_kernel<T, VEC, ITER, true, S, 1, WIN>>(p, sh, tensors, grid, s);
  return launch<ln_bwd_kernel<T, VEC, ITER, false, S, 1, WIN>>(p, sh, tensors, grid, s);
}
template <typename T, int VEC>
static int ln_launch_restore(const void *codes, const void *scales, const void *w, const void *b, int64_t T_, int d, void *n,
                             cudaStream_t s) {
  const int cols = d / VEC;
  int64_t step = ((int64_t)sm_count() * 8 * kRestoreThreads + cols - 1) / cols;   // eight blocks per SM, about
  if (step > T_) step = T_;
  const int64_t grid = (step * cols + kRestoreThreads - 1) / kRestoreThreads;
  ln_restore_kernel<T, VEC><<<(unsigned)grid, kRestoreThreads, 0, s>>>((const uint8_t *)codes, (const uint8_t *)scales,
                                                                       (const T *)w, (const T *)b, T_, d,
                                                                       (int)act8::blocks_of(d), step, (T *)n);
  MOE_CHECK_LAUNCH();
  return MOE_OK;
}

template <typename T, int VEC>
static int ln_launch_restore_windows(const void *codes, const void *scales, const void *w, const void *b, int64_t T_, int d, void *n,
                                     cudaStream_t s) {
  const int words = (d + 2 * VEC - 2) / VEC;
  int64_t step = ((int64_t)sm_count() * 8 * kRestoreThreads + words - 1) / words;   // eight blocks per SM, about
  step = (step + VEC - 1) / VEC * VEC;
  if (step > T_) step = T_;
  const int64_t grid = (step * words + kRestoreThreads - 1) / kRestoreThreads;
  ln_restore_windows_kernel<T, VEC><<<(unsigned)grid, kRestoreThreads, 0, s>>>(
      (const uint8_t *)codes, (const uint8_t *)scales, (const T *)w, (const T *)b, T_, d, (int)act8::blocks_of(d), words, step, (T *)n);
  MOE_CHECK_LAUNCH();
  return MOE_OK;
}

// Blocks of the backward: each leaves a partial row, so no more than the GPU holds at once (of a GB300's SMs, wherever the
// workspace's size is asked for).
static int ln_bwd_blocks(int64_t T, const Shape &s, int tensors) {
  int64_t b = 152 * per_sm(s, tensors, s.vec == 1 && s.iter <= 4 ? 2 * kMaxThreads : kMaxThreads);
  if (b > T) b = T;
  return b < 1 ? 1 : (int)b;
}

#define MOE_LN_DISPATCH(FN, WIN, ...)                                                                 \
  do {                                                                                                \
    if (dtype == MOE_BF16) {                                                                          \
      if (sh.vec == 8 && sh.iter == 1) rc = FN<__nv_bfloat16, 8, 1, WIN>(__VA_ARGS__);                \
      else if (sh.vec == 8) rc = FN<__nv_bfloat16, 8, 2, WIN>(__VA_ARGS__);                           \
      else if (sh.iter == 4) rc = FN<__nv_bfloat16, 1, 4, false>(__VA_ARGS__);                        \
      else rc = FN<__nv_bfloat16, 1, 16, false>(__VA_ARGS__);                                         \
    } else {                                                                                          \
      if (sh.vec == 4 && sh.iter == 1) rc = FN<float, 4, 1, WIN>(__VA_ARGS__);                        \
      else if (sh.vec == 4 && sh.iter == 2) rc = FN<float, 4, 2, WIN>(__VA_ARGS__);                   \
      else if (sh.vec == 4) rc = FN<float, 4, 4, WIN>(__VA_ARGS__);                                   \
      else if (sh.iter == 4) rc = FN<float, 1, 4, false>(__VA_ARGS__);                                \
      else rc = FN<float, 1, 16, false>(__VA_ARGS__);                                                 \
    }                                                                                                 \
  } while (0)

// How a call's rows are read: as vectors, as windows of them (where rows start anywhere, and there is enough for what the
// windows' weights and partial rows cost once per block), or value by value. Windows and values, in us: forward 500 x 333 bf16
// 3.1 and 2.8, 600 x 501 3.2 and 3.0, 300 x 1537 fp32 3.0 and 3.6, 150 x 4001 bf16 3.7 and 7.0, 8192 x 2047 24.8 and 49.1;
// restore 800 x 1537 fp32 4.3 and 4.2, 1023 x 1537 4.7 and 5.2, 8192 x 2047 bf16 15 and 35; backward 300 x 1537 fp32 (one row
// per block) 6.1 and 6.0, 650 x 1537 7.6 and 8.4, 8192 x 1537 35 and 52; 1300 x 501 bf16 (one row per block) 12.0 and 9.1, 3700
// x 501 (three) 12.9 and 12.9, 700 x 4001 (five) 15.9 and 14.5, 8192 x 2047 49 and 55.
constexpr int64_t kWindowsFwd = 400000, kWindowsRestore = 1500000;                         // values, more than
static int windows_bwd(int dtype) { return dtype == MOE_F32 ? 1 : 5; }                     // rows per block, more than
struct How {
  Shape sh;
  bool win;
};
static How how(int d, int dtype, bool may) {
  const Shape sh = shape_of(d, dtype);
  if (sh.vec > 1 || !may || d <= 32) return {sh, false};
  const Shape w = windows_of(d, dtype);
  return w.vec > 1 ? How{w, true} : How{sh, false};
}

}  // namespace norm
}  // namespace moe

using namespace moe;
using namespace moe::norm;

extern "C" size_t moe_layer_norm_bwd_workspace_size(int T, int d, int dtype) {
  if (T < 0 || d < 1 || d > MOE_NORM_MAX_D || (dtype != MOE_F32 && dtype != MOE_BF16)) return 0;
  int most = 0;
  for (int may = 0; may < 2; ++may)
    for (int tensors = 2; tensors <= 3; ++tensors) most = std::max(most, ln_bwd_blocks(T, how(d, dtype, may).sh, tensors));
  return (size_t)2 * most * d * sizeof(float) + 256;
}

extern "C" int moe_layer_norm_fwd(const void *x, const void *w, const void *b, int T, int d, int dtype, float eps, void *n,
                                  float *mean, float *rstd, void *codes, void *scales, moe_stream_t stream) {
  int rc = check_shape(T, d, dtype, eps);
  if (rc) return rc;
  if ((codes == nullptr) != (scales == nullptr)) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  if (bad(x) || bad(w) || bad(n) || !aligned16(b) || !aligned16(mean) || !aligned16(rstd) || !aligned16(codes) || !aligned16(scales))
    return MOE_ERR_INVALID_ARG;
  LnFwdParams p{};
  p.x = x;
  p.w = w;
  p.b = b;
  p.n = n;
  p.mean = mean;
  p.rstd = rstd;
  p.codes = (uint8_t *)codes;
  p.scales = (uint8_t *)scales;
  p.T = T;
  p.d = d;
  p.nb = (int)act8::blocks_of(d);
  p.eps = eps;
  const How h = how(d, dtype, (int64_t)T * d > kWindowsFwd);
  const Shape &sh = h.sh;
  if (h.win) MOE_LN_DISPATCH(ln_launch_fwd, true, p, sh, (cudaStream_t)stream);
  else MOE_LN_DISPATCH(ln_launch_fwd, false, p, sh, (cudaStream_t)stream);
  return rc;
}

extern "C" int moe_layer_norm_restore(const void *codes, const void *scales, const void *w, const void *b, int T, int d,
                                      int dtype, void *n, moe_stream_t stream) {
  int rc = check_shape(T, d, dtype, 1.0f);
  if (rc) return rc;
  if (T == 0) return MOE_OK;
  if (bad(codes) || bad(scales) || bad(w) || !aligned16(b) || bad(n)) return MOE_ERR_INVALID_ARG;
  cudaStream_t s = (cudaStream_t)stream;
  if (dtype == MOE_BF16 && d % act8::kBlock == 0) {
    const int cols = d / 16;
    int64_t step = ((int64_t)sm_count() * 8 * kRestoreThreads + cols - 1) / cols;   // eight blocks per SM, about
    if (step > T) step = T;
    const unsigned grid = (unsigned)((step * cols + kRestoreThreads - 1) / kRestoreThreads);
    ln_restore16_kernel<<<grid, kRestoreThreads, 0, s>>>((const uint4 *)codes, (const uint8_t *)scales, (const __nv_bfloat16 *)w,
                                                        (const __nv_bfloat16 *)b, T, d, step, ((uintptr_t)n & 31) == 0,
                                                        (__nv_bfloat16 *)n);
    MOE_CHECK_LAUNCH();
    return MOE_OK;
  }
  if (dtype == MOE_BF16) {
    if (d % 8 == 0) return ln_launch_restore<__nv_bfloat16, 8>(codes, scales, w, b, T, d, n, s);
    return (int64_t)T * d > kWindowsRestore ? ln_launch_restore_windows<__nv_bfloat16, 8>(codes, scales, w, b, T, d, n, s)
                           : ln_launch_restore<__nv_bfloat16, 1>(codes, scales, w, b, T, d, n, s);
  }
  if (d % 4 == 0) return ln_launch_restore<float, 4>(codes, scales, w, b, T, d, n, s);
  return (int64_t)T * d > kWindowsRestore ? ln_launch_restore_windows<float, 4>(codes, scales, w, b, T, d, n, s)
                         : ln_launch_restore<float, 1>(codes, scales, w, b, T, d, n, s);
}

extern "C" int moe_layer_norm_bwd(const void *dn, const void *x, const void *codes, const void *scales, const float *mean,
                                  const float *rstd, const void *w, const void *dx_in, int T, int d, int dtype, float eps,
                                  void *dx, void *dw, void *db, void *ws, size_t ws_bytes, moe_stream_t stream) {
  int rc = check_shape(T, d, dtype, eps);
  if (rc) return rc;
  if (bad(w) || bad(dw) || !aligned16(db) || bad(ws) || ((uintptr_t)ws & 255) ||
      ws_bytes < moe_layer_norm_bwd_workspace_size(T, d, dtype))
    return MOE_ERR_INVALID_ARG;
  const bool kept = codes != nullptr;
  if ((scales != nullptr) != kept || (kept && x)) return MOE_ERR_INVALID_ARG;
  if (T > 0 && (bad(dn) || bad(rstd) || bad(dx) || (dx_in && bad(dx_in)) ||
                (kept ? bad(codes) || bad(scales) : bad(x) || bad(mean))))
    return MOE_ERR_INVALID_ARG;
  LnBwdParams p{};
  p.dn = dn;
  p.x = x;
  p.dx_in = dx_in;
  p.w = w;
  p.mean = mean;
  p.rstd = rstd;
  p.codes = (const uint8_t *)codes;
  p.scales = (const uint8_t *)scales;
  p.dx = dx;
  p.part = static_cast<float *>(ws);
  p.T = T;
  p.d = d;
  p.nb = (int)act8::blocks_of(d);
  p.eps = eps;
  cudaStream_t s = (cudaStream_t)stream;
  How h = how(d, dtype, true);
  if (h.win && T <= (int64_t)windows_bwd(dtype) * ln_bwd_blocks(T, h.sh, dx_in ? 3 : 2)) h = how(d, dtype, false);
  Shape sh = h.sh;
  int rows = 1, grid = ln_bwd_blocks(T, sh, dx_in ? 3 : 2);
  // Two rows at a time where blocks have more rows than one: at T = 16384, d = 4096 bf16 86.8 against 89.0 us (from codes 84.7
  // against 91.0), at 8192 x 1024 fp32 18.8 against 21.4; not where bf16 rows are short enough for two blocks per SM: 26.8
  // against 25.7 at 8192 x 2048, 15.7 against 15.0 at 8192 x 1024.
  if (sh.vec > 1 && sh.iter == 1 && T > grid && d > 32 && (dtype == MOE_F32 || sh.threads > kMaxThreads / 2)) {
    rows = 2;
    grid = ln_bwd_blocks(T, sh, dx_in ? 6 : 4);
  }
  if (d <= 32) {   // one value per lane, in 64 bits
    sh.vec = sh.iter = 1;
    sh.threads = 32;
    sh.row_bytes = ((uint32_t)d * (uint32_t)dtype_size(dtype) + 15) / 16 * 16 + 16;
    if (dtype == MOE_BF16) rc = ln_launch_bwd<__nv_bfloat16, 1, 1, false, double>(p, sh, 1, grid, s);
    else rc = ln_launch_bwd<float, 1, 1, false, double>(p, sh, 1, grid, s);
  } else if (h.win) {
    MOE_LN_DISPATCH(ln_launch_bwd, true, p, sh, rows, grid, s);
  } else {
    MOE_LN_DISPATCH(ln_launch_bwd, false, p, sh, rows, grid, s);
  }
  if (rc) return rc;
  const dim3 g((d + 31) / 32, db ? 2 : 1);
  if (dtype == MOE_BF16) {
    using B = __nv_bfloat16;
    MOE_TRY_CUDA(launch_after(norm_bwd_sum_kernel<B>, g, dim3(1024), 0, s, (const float *)p.part, grid, d, (int)MOE_GATE_NONE,
                              (const B *)nullptr, (const B *)nullptr, (B *)dw, (B *)db, (B *)nullptr));
  } else {
    MOE_TRY_CUDA(launch_after(norm_bwd_sum_kernel<float>, g, dim3(1024), 0, s, (const float *)p.part, grid, d,
                              (int)MOE_GATE_NONE, (const float *)nullptr, (const float *)nullptr, (float *)dw, (float *)db,
                              (float *)nullptr));
  }
  return MOE_OK;
}
