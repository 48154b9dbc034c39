// One AdamW step over many tensors in one launch per kind of tensor, states in fp32 or in 8 bits.
//
//   m' = b1 m + (1 - b1) c g,   v' = b2 v + (1 - b2) (c g)^2,   c = grad_scale
//   p' = p (1 - lr wd) - lr (m' / (1 - b1^t)) / (sqrt(v' / (1 - b2^t)) + eps)
//
// HBM-bound: every value is read and written once. The tensors are cut into chunks of 4096 (8-bit states: 8192)
// values; a plan made on the host lists them, so a launch covers any number of tensors of any size and a block
// finds its tensor with two dependent loads. The bias corrections come from the step count in device
// memory, which the last block to have read it advances: a captured step counts on when it is replayed.
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
#include "f32x2.cuh"

namespace moe {
namespace adamw {

constexpr int kThreads = 256;
constexpr int kVec = 8;
constexpr int kBlockQ = MOE_ADAMW_BLOCK;
static_assert(kBlockQ == 32 * kVec, "a warp owns one block of an 8-bit state");

// Kinds of tensors: parameter and gradient type, fp32 master copy, state.
enum Kind { F32_F32 = 0, BF16_F32, BF16_MASTER_F32, F32_F8, BF16_F8, BF16_MASTER_F8, KINDS };

// Values per chunk. fp32 states: two passes of 8 values per thread. 8-bit states carry a third of the bytes per
// value, so four passes' loads are issued before any of them is used.
constexpr int chunk_of(int kind) { return kind >= F32_F8 ? 8192 : 4096; }

struct Chunk {
  int32_t tensor, index;          // values [index * chunk, ...) of the tensor
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

// e4m3 codes of y (|y| <= 448 but for rounding), rounded down in magnitude after adding u / 2^20 of a step, where
// u = h >> 12. z = y 2^-120 moves e4m3's exponents onto the lowest ones of fp32, subnormals onto subnormals, so
// its bits 20..26 are the code, adding u below them is the dither, and bit 31 is the sign.
__device__ __forceinline__ uint32_t dither(float z, uint32_t h) { return (h >> 12) + __float_as_uint(z); }
// Four codes from four such words, two at a time in 16-bit halves; at most 0x7e (448): a block's largest value may lie
// an ulp above it.
template <bool SIGNED> __device__ __forceinline__ uint32_t codes4(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  const uint32_t ab = __byte_perm(a, b, 0x7632), cd = __byte_perm(c, d, 0x7632);
  uint32_t p = __vminu2((ab << 4) & (SIGNED ? 0x7fff7fffu : 0xffffffffu), 0x7eff7effu);   // codes in bytes 1 and 3
  uint32_t q = __vminu2((cd << 4) & (SIGNED ? 0x7fff7fffu : 0xffffffffu), 0x7eff7effu);
  if (SIGNED) {
    p |= ab & 0x80008000u;
    q |= cd & 0x80008000u;
  }
  return __byte_perm(p, q, 0x7531);
}
// One code, of any y: a NaN or an infinity becomes e4m3 NaN.
__device__ __forceinline__ uint32_t code_any(float y, uint32_t h) {
  if (!(fabsf(y) <= 500.0f)) return 0x7fu;
  const uint32_t x = dither(y * 0x1p-120f, h);
  return min(x >> 20 & 0x7fu, 0x7eu) | (x >> 24 & 0x80u);
}
__device__ __forceinline__ float max_abs3(float a, float b, float c) {
  float r;
  asm("max.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// Approximate root: of subnormal numbers too, or (FTZ) taking them as zero. bf16 parameters with 8-bit states and no
// master use the second: the other costs them 4% (771 us against 740), and their v spans 2^36 within a block anyway.
template <bool FTZ> __device__ __forceinline__ float sqrt_approx(float v) {
  float r;
  if (FTZ) asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  else asm("sqrt.approx.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float rcp_approx(float v) {   // of normal numbers: eps or more
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
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

// Loads of values that are read once: they pass by the L1, which keeps the plan's entries.
__device__ __forceinline__ uint4 ld_once(const void *p) {
  uint4 r;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p));
  return r;
}
__device__ __forceinline__ uint2 ld_once2(const void *p) {
  uint2 r;
  asm volatile("ld.global.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(r.x), "=r"(r.y) : "l"(p));
  return r;
}
__device__ __forceinline__ void store8(float *p, const float *v) {
  reinterpret_cast<float4 *>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4 *>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
template <typename T> __device__ __forceinline__ float load1(const T *p) {
  if constexpr (sizeof(T) == 4) return *p;
  else return __bfloat162float(*p);
}

// Blocks per SM that the registers allow: a plan with at most that many chunks runs one chunk per block.
constexpr int per_sm_most(int kind) { return kind >= F32_F8 ? 2 : 3; }
// Blocks per SM on larger plans. Measured on one layer's 403M values (bf16): fp32 states with a master 1851 us at 2
// blocks, 1922 at 3, 1956 at 4. 8-bit states, (values per chunk, passes loaded ahead, blocks): (8192, 4, 2) 755 us,
// (8192, 4, 3) 795, (6144, 3, 3) 765, (4096, 2, 3) 800, (4096, 1, 5) 903, (4096, 1, 3) 1063; one fp32 per instruction
// instead of two: (4096, 1, 5) 934. Since then sums that are not paired (see update8) cost 18 us, scales that are written
// together took 37, and decay as a change of its own cost 7: 740.
constexpr int per_sm(int) { return 2; }
// 28 bytes per value (fp32 parameters, or bf16 ones with a master, and fp32 states): larger plans run one block per SM
// that loads a whole chunk, then writes it. As many bytes are in flight as with two blocks and one pass each, but HBM
// sees longer runs of reads and of writes. 201M values: 834 us against 905 with a master, 819 against 905 for fp32; from
// 460 chunks on it is ahead but for 2-9% around 900. The 22 bytes of bf16 parameters without a master are the
// other way round, 759 us against 673.
constexpr bool runs(int kind) { return kind == F32_F32 || kind == BF16_MASTER_F32; }

// The step's constants.
struct Coef {
  float lr, gs, lr1, inv_root2;
  uint32_t t32;
};

// One thread's eight values of a tensor as they lie in memory (the aligned, complete case).
template <int K> struct Raw8 {
  static constexpr bool kF8 = K >= F32_F8, kF32 = K == F32_F32 || K == F32_F8;
  static constexpr bool kMaster = K == BF16_MASTER_F32 || K == BF16_MASTER_F8;
  uint4 g[kF32 ? 2 : 1], p[kF32 || kMaster ? 2 : 1], m[kF8 ? 1 : 2], v[kF8 ? 1 : 2];
  float ms, vs;   // the block's scales (8-bit states)
  __device__ __forceinline__ void load(const Tensor &t, int64_t i0) {
    const int64_t es = kF32 ? 4 : 2;
    const uint8_t *gp = (const uint8_t *)t.g + i0 * es;
    g[0] = ld_once(gp);
    if (kF32) g[kF32 ? 1 : 0] = ld_once(gp + 16);
    const uint8_t *pp = kMaster ? (const uint8_t *)(t.master + i0) : (const uint8_t *)t.p + i0 * es;
    p[0] = ld_once(pp);
    if (kF32 || kMaster) p[kF32 || kMaster ? 1 : 0] = ld_once(pp + 16);
    if (kF8) {
      const uint2 a = ld_once2((const uint8_t *)t.m + i0), b = ld_once2((const uint8_t *)t.v + i0);
      m[0] = make_uint4(a.x, a.y, 0, 0);
      v[0] = make_uint4(b.x, b.y, 0, 0);
    } else {
      const float *mp = (const float *)t.m + i0, *vp = (const float *)t.v + i0;
      m[0] = ld_once(mp);
      m[kF8 ? 0 : 1] = ld_once(mp + 4);
      v[0] = ld_once(vp);
      v[kF8 ? 0 : 1] = ld_once(vp + 4);
    }
  }
};
__device__ __forceinline__ void unpack_f32x8(const uint4 &a, const uint4 &b, float *v) {
  v[0] = __uint_as_float(a.x); v[1] = __uint_as_float(a.y); v[2] = __uint_as_float(a.z); v[3] = __uint_as_float(a.w);
  v[4] = __uint_as_float(b.x); v[5] = __uint_as_float(b.y); v[6] = __uint_as_float(b.z); v[7] = __uint_as_float(b.w);
}

// Eight values of a tensor, the thread's own from i0 on. FULL: all eight are inside it, vector access is aligned and
// `raw` holds them; otherwise the `live` ones inside are read one by one. All lanes of a warp take part (8-bit
// states: its 256 values are one block, whose scales raw.ms and raw.vs are replaced by the new ones).
template <int K, bool FULL>
__device__ __forceinline__ void update8(const Tensor &t, Raw8<K> &raw, int64_t i0, int live, const Hyper &hy,
                                        const Coef &co, float decay) {
  constexpr bool kF8 = K >= F32_F8;
  constexpr bool kMaster = K == BF16_MASTER_F32 || K == BF16_MASTER_F8;
  constexpr bool kF32 = K == F32_F32 || K == F32_F8;
  // 8-bit states of an fp32 parameter (or master): every root is rounded to nearest and y before it is moved, so codes are
  // those of the formulas bit for bit. A code on the other side of a rounding threshold (one in a million
  // otherwise) changes the next update by a step of v; bf16 parameters hide that, fp32 ones show it. Here it costs
  // nothing (HBM has 16 bytes to move per value); without a master it takes 740 us to 897.
  constexpr bool kExact = K == F32_F8 || K == BF16_MASTER_F8;
  using T = typename std::conditional<kF32, float, __nv_bfloat16>::type;
  const T *gp = (const T *)t.g + i0;
  T *pp = (T *)t.p + i0;
  float *master = t.master + (kMaster ? i0 : 0);
  float *mf = (float *)t.m + (kF8 ? 0 : i0), *vf = (float *)t.v + (kF8 ? 0 : i0);
  uint8_t *m8 = (uint8_t *)t.m + (kF8 ? i0 : 0), *v8 = (uint8_t *)t.v + (kF8 ? i0 : 0);
  float g[kVec], p[kVec], m[kVec], v[kVec];
  if (FULL) {
    if (kF32) unpack_f32x8(raw.g[0], raw.g[kF32 ? 1 : 0], g);
    else unpack_bf16x8(raw.g[0], g);
    if (kF32 || kMaster) unpack_f32x8(raw.p[0], raw.p[kF32 || kMaster ? 1 : 0], p);
    else unpack_bf16x8(raw.p[0], p);
    if (kF8) {
      unpack_e4m3x8(make_uint2(raw.m[0].x, raw.m[0].y), m);
      unpack_e4m3x8(make_uint2(raw.v[0].x, raw.v[0].y), v);
    } else {
      unpack_f32x8(raw.m[0], raw.m[kF8 ? 0 : 1], m);
      unpack_f32x8(raw.v[0], raw.v[kF8 ? 0 : 1], v);
    }
  } else {
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
      g[j] = p[j] = m[j] = v[j] = 0.0f;
      if (j >= live) continue;
      g[j] = load1(gp + j);
      p[j] = kMaster ? master[j] : load1(pp + j);
      m[j] = kF8 ? (float)((const __nv_fp8_e4m3 *)m8)[j] : mf[j];
      v[j] = kF8 ? (float)((const __nv_fp8_e4m3 *)v8)[j] : vf[j];
    }
  }
  const uint32_t h0 = weyl((uint32_t)i0, co.t32);
  float sum = 0.0f;   // of the parameters: NaN where one of them is
  bool odd = false;
  if constexpr (!kF8) {
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
      const float gj = g[j] * co.gs;
      m[j] = fmaf(hy.beta1, m[j], hy.omb1 * gj);
      v[j] = fmaf(hy.beta2, v[j], hy.omb2 * gj * gj);
      // approximate root and reciprocal: off by a few 2^-24, on a term that is a small part of p
      p[j] += fmaf(p[j], decay, co.lr1 * m[j] * rcp_approx(fmaf(sqrt_approx<false>(v[j]), co.inv_root2, hy.eps)));
      sum += p[j];
    }
    odd = sum != sum;
    if (FULL) {
      store8(mf, m);
      store8(vf, v);
    } else {
#pragma unroll
      for (int j = 0; j < kVec; ++j) {
        if (j >= live) continue;
        mf[j] = m[j];
        vf[j] = v[j];
      }
    }
  } else {
    // m and v are rounded at each operation (no fused multiply-add), and the largest root is the root of the
    // largest v, rounded to nearest: the scales then follow from the formulas alone, bit for bit, and a
    // block's largest value gets the code it should. The other roots may be approximate (but for kExact).
    const F2 b1 = pair(hy.beta1, hy.beta1), b2 = pair(hy.beta2, hy.beta2), ms2 = pair(raw.ms, raw.ms), vs2 = pair(raw.vs, raw.vs);
    const float kg1 = hy.omb1 * co.gs, kg2 = hy.omb2 * (co.gs * co.gs);
    const F2 c1 = pair(kg1, kg1), c2 = pair(kg2, kg2);
    F2 m2[kVec / 2];
    float mx = 0.0f, vx = 0.0f;
#pragma unroll
    for (int j = 0; j < kVec / 2; ++j) {
      const F2 gg = pair(g[2 * j], g[2 * j + 1]);
      // the sums one value at a time: the assembler fuses a paired product and sum
      float x, y, x1, y1;
      split(mul(b1, mul(pair(m[2 * j], m[2 * j + 1]), ms2)), x, y);
      split(mul(c1, gg), x1, y1);
      m[2 * j] = __fadd_rn(x, x1);
      m[2 * j + 1] = __fadd_rn(y, y1);
      const F2 a = mul(pair(v[2 * j], v[2 * j + 1]), vs2);
      split(mul(b2, mul(a, a)), x, y);
      split(mul(c2, mul(gg, gg)), x1, y1);
      v[2 * j] = __fadd_rn(x, x1);
      v[2 * j + 1] = __fadd_rn(y, y1);
      m2[j] = pair(m[2 * j], m[2 * j + 1]);
      mx = max_abs3(m[2 * j], m[2 * j + 1], mx);
      vx = max_abs3(v[2 * j], v[2 * j + 1], vx);
    }
    mx = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(mx)));   // of numbers >= 0, as integers
    const float vtop = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(vx)));
    vx = sqrtf(vtop);
    const F2 ir = pair(co.inv_root2, co.inv_root2), eps = pair(hy.eps, hy.eps), l1 = pair(co.lr1, co.lr1), dc = pair(decay, decay);
    F2 sum2 = pair(0.0f, 0.0f);
#pragma unroll
    for (int j = 0; j < kVec / 2; ++j) {
      if (kExact) {
        v[2 * j] = sqrtf(v[2 * j]);
        v[2 * j + 1] = sqrtf(v[2 * j + 1]);
      } else {
        v[2 * j] = v[2 * j] == vtop ? vx : sqrt_approx<true>(v[2 * j]);
        v[2 * j + 1] = v[2 * j + 1] == vtop ? vx : sqrt_approx<true>(v[2 * j + 1]);
      }
      float d0, d1;
      split(fma(pair(v[2 * j], v[2 * j + 1]), ir, eps), d0, d1);
      // the reciprocal is approximate, as above
      const F2 p0 = pair(p[2 * j], p[2 * j + 1]), pp = add(p0, fma(p0, dc, mul(mul(l1, m2[j]), pair(rcp_approx(d0), rcp_approx(d1)))));
      sum2 = add(sum2, pp);
      split(pp, p[2 * j], p[2 * j + 1]);
    }
    float s0, s1;
    split(sum2, s0, s1);
    sum = s0 + s1;
    // A NaN in m or v shows in p and so in the sum; infinities show in the maxima. Such blocks, and those whose
    // scaling would leave fp32's normal range, take the general form.
    odd = __any_sync(0xffffffffu, sum != sum) || !(fmaxf(mx, vx) < 16384.0f);
    if (odd) {   // a non-finite value counts for nothing in the scale and is held as NaN
      constexpr float kMax = 3.402823466e38f;
      mx = vx = 0.0f;
#pragma unroll
      for (int j = 0; j < kVec; ++j) {
        if (fabsf(m[j]) <= kMax) mx = fmaxf(mx, fabsf(m[j]));
        if (v[j] <= kMax) vx = fmaxf(vx, v[j]);
      }
      mx = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(mx)));
      vx = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(vx)));
    }
    // below 1e-30 a block is held as zeros
    const bool mk = mx >= 1e-30f, vk = vx >= 1e-30f;
    const float mi = mk ? __frcp_rn(mx) * 448.0f : 0.0f, vi = vk ? __frcp_rn(vx) * 448.0f : 0.0f;
    uint32_t mc[2], vc[2];   // four codes each
    if (!odd) {
      // kExact: y is rounded, and its move onto fp32's lowest exponents (see dither) then drops what lies below 2^-20 of
      // a code's smallest step. Otherwise one product does both.
      const F2 mi2 = pair(mi, mi), vi2 = pair(vi, vi), low = pair(0x1p-120f, 0x1p-120f);
      const F2 mz2 = mul(mi2, low), vz2 = mul(vi2, low);
      uint32_t mw[kVec], vw[kVec];
#pragma unroll
      for (int j = 0; j < kVec; j += 2) {
        const uint32_t h = h0 + (uint32_t)j * 2654435769u, h1 = h0 + (uint32_t)(j + 1) * 2654435769u;
        float x, y;
        split(kExact ? mul_rz(mul(m2[j / 2], mi2), low) : mul(m2[j / 2], mz2), x, y);
        mw[j] = dither(x, h);
        mw[j + 1] = dither(y, h1);
        split(kExact ? mul_rz(mul(pair(v[j], v[j + 1]), vi2), low) : mul(pair(v[j], v[j + 1]), vz2), x, y);
        vw[j] = dither(x, h + 0x55555555u);
        vw[j + 1] = dither(y, h1 + 0x55555555u);
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        mc[j] = codes4<true>(mw[4 * j], mw[4 * j + 1], mw[4 * j + 2], mw[4 * j + 3]);
        vc[j] = codes4<false>(vw[4 * j], vw[4 * j + 1], vw[4 * j + 2], vw[4 * j + 3]);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        mc[j] = vc[j] = 0;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const uint32_t h = h0 + (uint32_t)(4 * j + q) * 2654435769u;
          mc[j] |= code_any(m[4 * j + q] * mi, h) << (8 * q);
          vc[j] |= code_any(v[4 * j + q] * vi, h + 0x55555555u) << (8 * q);
        }
      }
    }
    raw.ms = mk ? mx * (1.0f / 448.0f) : 0.0f;
    raw.vs = vk ? vx * (1.0f / 448.0f) : 0.0f;
    if (FULL) {
      *reinterpret_cast<uint2 *>(m8) = make_uint2(mc[0], mc[1]);
      *reinterpret_cast<uint2 *>(v8) = make_uint2(vc[0], vc[1]);
    } else {
#pragma unroll
      for (int j = 0; j < kVec; ++j) {
        if (j >= live) continue;
        m8[j] = (uint8_t)(mc[j / 4] >> (8 * (j & 3)));
        v8[j] = (uint8_t)(vc[j / 4] >> (8 * (j & 3)));
      }
    }
  }
  if constexpr (kF32) {
    if (FULL) {
      store8(pp, p);
    } else {
#pragma unroll
      for (int j = 0; j < kVec; ++j)
        if (j < live) pp[j] = p[j];
    }
  } else {
    uint32_t pb[kVec / 2];   // two bf16 each
    if (kMaster) {
#pragma unroll
      for (int j = 0; j < kVec / 2; ++j) pb[j] = pack_bf16x2(p[2 * j], p[2 * j + 1]);
    } else {
#pragma unroll
      for (int j = 0; j < kVec; j += 2) {
        uint32_t b[2];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          b[q] = ((h0 + 0xaaaaaaaau + (uint32_t)(j + q) * 2654435769u) >> 16) + __float_as_uint(p[j + q]);
          if (odd && p[j + q] != p[j + q]) b[q] = 0x7fff0000u;   // the sum can wrap on the bits of a NaN
        }
        pb[j / 2] = __byte_perm(b[0], b[1], 0x7632);
      }
    }
    if (FULL) {
      *reinterpret_cast<uint4 *>(pp) = make_uint4(pb[0], pb[1], pb[2], pb[3]);
      if (kMaster) store8(master, p);
    } else {
#pragma unroll
      for (int j = 0; j < kVec; ++j) {
        if (j >= live) continue;
        pp[j] = __ushort_as_bfloat16((unsigned short)(pb[j / 2] >> (16 * (j & 1))));
        if (kMaster) master[j] = p[j];
      }
    }
  }
}

// LARGE: the plan has more chunks than blocks run at once, and runs(K).
template <int K, bool LARGE>
__global__ void __launch_bounds__(kThreads, LARGE ? 1 : per_sm_most(K))
    adamw_kernel(const Tensor *__restrict__ tensors, const Chunk *__restrict__ chunks, int64_t nchunks, const Hyper hy,
                 moe_adamw_state *st, int bump) {
  constexpr bool kF8 = K >= F32_F8;
  constexpr int kChunk = chunk_of(K), kPasses = kChunk / (kThreads * kVec);
  const int lane = threadIdx.x & 31;
  Chunk ahead = blockIdx.x < nchunks ? chunks[blockIdx.x] : Chunk{0, 0};
  const int64_t step = st->step + 1;
  Coef co;
  co.lr = st->lr;
  co.gs = st->grad_scale;
  // Every thread of a block has read the step when the block arrives (the vote needs its value, so no load of it is
  // still on its way), and the block that arrives last may advance it at once. (Arriving at the kernel's end put a fence
  // and an atomic behind the last stores.)
  __syncthreads_or(step <= 0);
  if (bump && threadIdx.x == 0 && atomicAdd(&st->arrived, 1u) == gridDim.x - 1) {
    st->arrived = 0;
    st->step = step;
  }
  const float bc1 = -expm1f((float)step * hy.log_beta1), bc2 = -expm1f((float)step * hy.log_beta2);
  co.lr1 = -co.lr / bc1;
  co.inv_root2 = 1.0f / sqrtf(bc2);
  co.t32 = (uint32_t)step;

  for (int64_t ci = blockIdx.x; ci < nchunks; ci += gridDim.x) {
    const Chunk ch = ahead;
    if (ci + gridDim.x < nchunks) ahead = chunks[ci + gridDim.x];
    const Tensor t = tensors[ch.tensor];
    // The change that decay makes, not the factor 1 - lr wd: fp32 numbers just below 1 are 6e-8 apart, so 1e-7
    // would act as 1.2e-7 on every value alike, and half of that not at all.
    const float decay = -co.lr * t.weight_decay;
    const int64_t first = (int64_t)ch.index * kChunk + threadIdx.x * kVec;
    if (t.aligned && (int64_t)(ch.index + 1) * kChunk <= t.n) {
      if constexpr (kF8) {
        // A warp takes kPasses blocks in a row, all their loads first. One lane each carries their scales, which are
        // written together: single words, two for every 256 values, cost 37 us on 403M values.
        const int64_t i0 = (int64_t)ch.index * kChunk + (threadIdx.x >> 5) * (kPasses * kBlockQ) + lane * kVec;
        float *scales = (lane < kPasses ? t.m_scale : t.v_scale) + i0 / kBlockQ + (lane & (kPasses - 1));
        float scale = lane < 2 * kPasses ? *scales : 0.0f;
        Raw8<K> r[kPasses];
#pragma unroll
        for (int a = 0; a < kPasses; ++a) r[a].load(t, i0 + a * kBlockQ);
#pragma unroll
        for (int a = 0; a < kPasses; ++a) {
          r[a].ms = __shfl_sync(0xffffffffu, scale, a);
          r[a].vs = __shfl_sync(0xffffffffu, scale, kPasses + a);
          update8<K, true>(t, r[a], i0 + a * kBlockQ, kVec, hy, co, decay);
          if (lane == a) scale = r[a].ms;
          if (lane == kPasses + a) scale = r[a].vs;
        }
        if (lane < 2 * kPasses) *scales = scale;
      } else if constexpr (LARGE) {
        Raw8<K> r[kPasses];
#pragma unroll
        for (int a = 0; a < kPasses; ++a) r[a].load(t, first + a * (kThreads * kVec));
#pragma unroll
        for (int a = 0; a < kPasses; ++a) update8<K, true>(t, r[a], first + a * (kThreads * kVec), kVec, hy, co, decay);
      } else {
#pragma unroll 1
        for (int pass = 0; pass < kPasses; ++pass) {
          Raw8<K> raw;
          raw.load(t, first + pass * (kThreads * kVec));
          update8<K, true>(t, raw, first + pass * (kThreads * kVec), kVec, hy, co, decay);
        }
      }
    } else {
#pragma unroll 1
      for (int pass = 0; pass < kPasses; ++pass) {
        const int64_t i0 = first + pass * (kThreads * kVec);
        const int64_t left = t.n - i0, warp_left = left + lane * kVec;
        if (warp_left <= 0) break;
        Raw8<K> raw;
        if (kF8) {
          raw.ms = t.m_scale[i0 / kBlockQ];
          raw.vs = t.v_scale[i0 / kBlockQ];
        }
        // 8-bit states: the warp's 256 values are updated together
        if (t.aligned && (kF8 ? warp_left >= 32 * kVec : left >= kVec)) {
          raw.load(t, i0);
          update8<K, true>(t, raw, i0, kVec, hy, co, decay);
        } else {
          update8<K, false>(t, raw, i0, left >= kVec ? kVec : (left > 0 ? (int)left : 0), hy, co, decay);
        }
        if (kF8 && lane == 0) {
          t.m_scale[i0 / kBlockQ] = raw.ms;
          t.v_scale[i0 / kBlockQ] = raw.vs;
        }
      }
    }
  }
}

static int kind_of(const moe_adamw_tensor &t) {
  const int base = t.dtype == MOE_F32 ? 0 : (t.master ? 2 : 1);
  return base + (t.state == MOE_ADAMW_F8 ? 3 : 0);
}

static int64_t chunks_of(const moe_adamw_tensor &t) {
  const int c = chunk_of(kind_of(t));
  return t.n > 0 ? (t.n - 1) / c + 1 : 0;
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
  if (chunks_of(t) >= ((int64_t)1 << 31)) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

template <int K>
static int launch(const uint8_t *dev, const Header *h, int64_t first, int64_t n, const Hyper &hy, moe_adamw_state *st,
                  bool bump, cudaStream_t s) {
  const int sms = sm_count();
  const bool small = n <= (int64_t)sms * per_sm_most(K);
  const int64_t grid = small ? (n < 1 ? 1 : n) : (int64_t)sms * (runs(K) ? 1 : per_sm(K));
  const Tensor *tensors = (const Tensor *)(dev + sizeof(Header));
  const Chunk *chunks = (const Chunk *)(dev + h->chunks_at) + first;
  if (runs(K) && !small)
    adamw_kernel<K, runs(K)><<<(int)grid, kThreads, 0, s>>>(tensors, chunks, n, hy, st, bump ? 1 : 0);
  else
    adamw_kernel<K, false><<<(int)grid, kThreads, 0, s>>>(tensors, chunks, n, hy, st, bump ? 1 : 0);
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
  for (int i = 0; i < count; ++i) chunks += (size_t)chunks_of(tensors[i]);
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
      const int64_t n = chunks_of(tensors[i]);
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
  if (!(beta1 >= 0.0 && beta1 < 1.0) || !(beta2 >= 0.0 && beta2 < 1.0) || !(eps >= 0x1p-126f)) return MOE_ERR_INVALID_ARG;
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
