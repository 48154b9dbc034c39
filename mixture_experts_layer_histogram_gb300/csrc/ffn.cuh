// What the kernels of the gated feed-forward block share (ffn*.cu): the gate's arithmetic and the host entry points.
//
//   a = x Wg^T, b = x Wu^T, h = act(a) b, y = h Wd^T
//
// Both gates are act(a) = a s, s = sigma(g(a)) with a cubic g: silu g = a, gelu (its tanh form, 0.5 a (1 + tanh(c (a +
// 0.044715 a^3))), c = sqrt(2 / pi)) g = 2 c (a + 0.044715 a^3), since 0.5 (1 + tanh(v)) = sigma(2 v). So one code
// path serves both: g = a (k0 + k1 a^2), act' = s + a s (1 - s) (k0 + 3 k1 a^2).
#pragma once

#include "act8.cuh"
#include "common.cuh"
#include "f32x2.cuh"

namespace moe {
namespace ffn {

struct Gate {
  float k0, k1;
};
inline Gate gate_of(int act) {
  const float c2 = 1.5957691216057308f;   // 2 sqrt(2 / pi)
  return act == MOE_ACT_GELU ? Gate{c2, c2 * 0.044715f} : Gate{1.0f, 0.0f};
}

// sigma(z) for the bf16 outputs (sigmoidf_), and with full fp32 accuracy for fp32 ones
template <bool EXACT> __device__ __forceinline__ float sigma(float z) {
  if (EXACT) return 1.0f / (1.0f + expf(-z));
  return sigmoidf_(z);
}
// a^2, held below infinity: times k1 = 0 it has to stay 0, and at 1e30 the sigmoid has long been 0 or 1
__device__ __forceinline__ float square_of(float a) { return fminf(a * a, 1e30f); }
template <bool EXACT = false> __device__ __forceinline__ float gated(float a, const Gate &k) {
  return a * sigma<EXACT>(a * fmaf(k.k1, square_of(a), k.k0));
}
// act(a) and act'(a), in full fp32
__device__ __forceinline__ void gate_and_slope(float a, const Gate &k, float &act, float &slope) {
  const float q = square_of(a), s = sigma<true>(a * fmaf(k.k1, q, k.k0));
  act = a * s;
  slope = fmaf(act * (1.0f - s), fmaf(3.0f * k.k1, q, k.k0), s);
}

// The same for two values at a time, for the bf16 epilogues, whose instructions have to hide behind the products. The silu gate
// leaves the cubic out (its k1 is 0): k.k1 is the same in all threads, so that is one branch.
__device__ __forceinline__ F2 both(float v) { return pair(v, v); }
__device__ __forceinline__ F2 sigma2(F2 z) {   // 1 / (1 + 2^(-z log2 e)): ex2 and rcp, each good to an ulp or two
  float x, y;
  split(mul(z, both(-1.4426950408889634f)), x, y);
  asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(x));
  asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(y));
  split(add(pair(x, y), both(1.0f)), x, y);
  asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(x));
  asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(y));
  return pair(x, y);
}
__device__ __forceinline__ F2 square2(F2 a) {   // square_of
  float x, y;
  split(mul(a, a), x, y);
  return pair(fminf(x, 1e30f), fminf(y, 1e30f));
}
template <bool CUBIC> __device__ __forceinline__ F2 gated2(F2 a, const Gate &k) {
  return mul(a, sigma2(CUBIC ? mul(a, fma(both(k.k1), square2(a), both(k.k0))) : a));
}
template <bool CUBIC> __device__ __forceinline__ void gate_and_slope2(F2 a, const Gate &k, F2 &act, F2 &slope) {
  if (CUBIC) {
    const F2 q = square2(a), s = sigma2(mul(a, fma(both(k.k1), q, both(k.k0))));
    act = mul(a, s);
    slope = fma(mul(act, fma(s, both(-1.0f), both(1.0f))), fma(both(3.0f * k.k1), q, both(k.k0)), s);
  } else {
    const F2 s = sigma2(a);
    act = mul(a, s);
    slope = fma(act, fma(s, both(-1.0f), both(1.0f)), s);
  }
}

// One call's sizes and buffers (see moe.h). bf16 and fp32 share it.
struct Block {
  int T, d, f;
  Gate gate;
  const void *x, *w_gate_up, *w_down, *add;   // add: y_in, or dx_in
  void *ab;                                   // [T, 2f] in dtype, or 8-bit codes with `scales`; null: not kept
  uint8_t *scales;
  void *h, *y;
  const void *dy;
  void *dab, *dx, *dw_gate_up, *dw_down;
  WsHeader *hdr;
  void *ws;                                   // past the header
};

// bf16, tensor cores (ffn_gemm.cu)
size_t gemm_workspace(int T, int d, int f, bool backward);
int gemm_fwd(const Block &b, cudaStream_t s);
int gemm_bwd(const Block &b, cudaStream_t s);
// bf16, few tokens: forward that keeps nothing (ffn_few.cu)
constexpr int kFewTokens = 64;
bool few_ring(int T, int d, int f);   // whether it streams the weights through its ring
int few_fwd(const Block &b, cudaStream_t s);
// fp32 (ffn_f32.cu)
int f32_fwd(const Block &b, cudaStream_t s);
int f32_bwd(const Block &b, cudaStream_t s);

}  // namespace ffn
}  // namespace moe
