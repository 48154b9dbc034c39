// The gated feed-forward block in true fp32 (FFMA on the CUDA cores; tf32 tensor cores would not hold fp32), any sizes.
//
// One kernel for the five products: C[m, n] = sum_k A(m, k) B(n, k), operands addressed by strides (K-major and MN-major alike), a
// tile of 128 x 128 (64 x 64 where that leaves SMs idle), 16-deep steps through two buffers in shared memory, the
// next step's loads in registers while this one is multiplied, two fp32 per instruction. A thread's columns lie in the two halves of
// the tile, so GATEUP takes gate rows for the first half and the same features' up rows for the second, and a thread
// holds a and b of the same features.
#include "f32x2.cuh"
#include "ffn.cuh"

namespace moe {
namespace ffn {
namespace simt {

enum Kind { GATEUP = 0, PLAIN = 1, DH = 2 };

constexpr int BK = 16, THREADS = 256;

struct Args {
  const float *A, *B;
  int64_t am, ak, bn, bk;    // strides
  int M, N, K;               // N: columns of B's rows (GATEUP, DH: f)
  float *C;                  // GATEUP kept ab (null: not kept); DH dab; PLAIN the result
  float *C2;                 // GATEUP h
  const float *in;           // DH kept ab; PLAIN what is added (null: nothing)
  Gate gate;
};

// TM: rows and columns per thread; the tile is 16 TM square.
template <int KIND, int TM>
__global__ void __launch_bounds__(THREADS) ffn_f32_kernel(const Args p) {
  constexpr int BM = 16 * TM, G = TM / 2, PER = BM * BK / THREADS, LD = BM + 4;
  __shared__ __align__(16) float As[2][BK][LD], Bs[2][BK][LD];
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int m0 = blockIdx.y * BM, n0 = blockIdx.x * (KIND == GATEUP ? BM / 2 : BM);
  float ra[PER], rb[PER];
  // Element i of this thread: consecutive threads along the axis whose stride is 1
  const bool a_k = p.ak == 1, b_k = p.bk == 1;
  auto place = [&](int i, bool along_k, int &r, int &k) {
    const int e = i * THREADS + threadIdx.x;
    k = along_k ? e % BK : e / BM;
    r = along_k ? e / BK : e % BM;
  };
  auto load = [&](int k0) {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      int r, k;
      place(i, a_k, r, k);
      ra[i] = m0 + r < p.M && k0 + k < p.K ? p.A[(m0 + r) * p.am + (k0 + k) * p.ak] : 0.0f;
      place(i, b_k, r, k);
      int64_t row = n0 + r;
      bool ok = row < p.N;
      if (KIND == GATEUP && r >= BM / 2) {
        ok = n0 + r - BM / 2 < p.N;
        row = (int64_t)p.N + n0 + r - BM / 2;
      }
      rb[i] = ok && k0 + k < p.K ? p.B[row * p.bn + (k0 + k) * p.bk] : 0.0f;
    }
  };
  auto stash = [&](int b) {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      int r, k;
      place(i, a_k, r, k);
      As[b][k][r] = ra[i];
      place(i, b_k, r, k);
      Bs[b][k][r] = rb[i];
    }
  };
  F2 acc[TM][TM / 2];
#pragma unroll
  for (int i = 0; i < TM; ++i) {
#pragma unroll
    for (int j = 0; j < TM / 2; ++j) acc[i][j] = pair(0.0f, 0.0f);
  }
  load(0);
  stash(0);
  __syncthreads();
  const int steps = (p.K + BK - 1) / BK;
  for (int s = 0; s < steps; ++s) {
    const int b = s & 1;
    if (s + 1 < steps) load((s + 1) * BK);
#pragma unroll
    for (int k = 0; k < BK; ++k) {
      float a[TM];
      F2 bb[TM / 2];
#pragma unroll
      for (int i = 0; i < TM; ++i) a[i] = As[b][k][(i / G) * (BM / 2) + ty * G + i % G];
#pragma unroll
      for (int j = 0; j < TM / 2; ++j)
        bb[j].v = *reinterpret_cast<const uint64_t *>(&Bs[b][k][(2 * j / G) * (BM / 2) + tx * G + 2 * j % G]);
#pragma unroll
      for (int i = 0; i < TM; ++i) {
        const F2 aa = pair(a[i], a[i]);
#pragma unroll
        for (int j = 0; j < TM / 2; ++j) acc[i][j] = fma(aa, bb[j], acc[i][j]);
      }
    }
    if (s + 1 < steps) stash(b ^ 1);   // the buffer that everyone left at the barrier of the step before
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < TM; ++i) {
    const int64_t m = m0 + (i / G) * (BM / 2) + ty * G + i % G;
    if (m >= p.M) continue;
    float v[TM];
#pragma unroll
    for (int j = 0; j < TM / 2; ++j) split(acc[i][j], v[2 * j], v[2 * j + 1]);
#pragma unroll
    for (int j = 0; j < (KIND == GATEUP ? G : TM); ++j) {
      const int64_t n = n0 + (j / G) * (BM / 2) + tx * G + j % G;
      if (n >= p.N) continue;
      if (KIND == GATEUP) {
        const float a = v[j], b = v[j + G];
        if (p.C) {
          p.C[m * 2 * p.N + n] = a;
          p.C[m * 2 * p.N + p.N + n] = b;
        }
        p.C2[m * p.N + n] = gated<true>(a, p.gate) * b;
      } else if (KIND == DH) {
        const float a = p.in[m * 2 * p.N + n], b = p.in[m * 2 * p.N + p.N + n];
        float act, slope;
        gate_and_slope<true>(a, p.gate, act, slope);
        p.C[m * 2 * p.N + n] = v[j] * b * slope;
        p.C[m * 2 * p.N + p.N + n] = v[j] * act;
      } else {
        p.C[m * p.N + n] = v[j] + (p.in ? p.in[m * p.N + n] : 0.0f);
      }
    }
  }
}

template <int KIND> static int launch(const Args &a, cudaStream_t s) {
  const auto blocks = [&](int bm) {
    const int bn = KIND == GATEUP ? bm / 2 : bm;
    return dim3((unsigned)((a.N + bn - 1) / bn), (unsigned)((a.M + bm - 1) / bm));
  };
  const dim3 big = blocks(128);
  if (big.y > 65535u) return MOE_ERR_UNSUPPORTED;
  if ((int64_t)big.x * big.y >= sm_count()) {
    ffn_f32_kernel<KIND, 8><<<big, THREADS, 0, s>>>(a);
  } else {
    ffn_f32_kernel<KIND, 4><<<blocks(64), THREADS, 0, s>>>(a);
  }
  MOE_CHECK_LAUNCH();
  return MOE_OK;
}

}  // namespace simt

using simt::Args;

int f32_fwd(const Block &b, cudaStream_t s) {
  Args a{};
  a.A = (const float *)b.x; a.am = b.d; a.ak = 1;
  a.B = (const float *)b.w_gate_up; a.bn = b.d; a.bk = 1;
  a.M = b.T; a.N = b.f; a.K = b.d;
  a.C = (float *)b.ab; a.C2 = (float *)b.h;
  a.gate = b.gate;
  const int rc = simt::launch<simt::GATEUP>(a, s);
  if (rc) return rc;
  a.A = (const float *)b.h; a.am = b.f;
  a.B = (const float *)b.w_down; a.bn = b.f;
  a.N = b.d; a.K = b.f;
  a.C = (float *)b.y; a.in = (const float *)b.add;
  return simt::launch<simt::PLAIN>(a, s);
}

int f32_bwd(const Block &b, cudaStream_t s) {
  const int64_t f = b.f, d = b.d;
  Args a{};
  a.gate = b.gate;
  a.A = (const float *)b.dy; a.am = d; a.ak = 1;                 // dh = dy Wd
  a.B = (const float *)b.w_down; a.bn = 1; a.bk = f;
  a.M = b.T; a.N = b.f; a.K = b.d;
  a.in = (const float *)b.ab; a.C = (float *)b.dab;
  int rc = simt::launch<simt::DH>(a, s);
  if (rc) return rc;
  a.A = (const float *)b.dab; a.am = 2 * f; a.ak = 1;            // dx = dab Wgu
  a.B = (const float *)b.w_gate_up; a.bn = 1; a.bk = d;
  a.N = b.d; a.K = 2 * b.f;
  a.in = (const float *)b.add; a.C = (float *)b.dx;
  if ((rc = simt::launch<simt::PLAIN>(a, s))) return rc;
  a.A = (const float *)b.dy; a.am = 1; a.ak = d;                 // dWd = dy^T h
  a.B = (const float *)b.h; a.bn = 1; a.bk = f;
  a.M = b.d; a.N = b.f; a.K = b.T;
  a.in = nullptr; a.C = (float *)b.dw_down;
  if ((rc = simt::launch<simt::PLAIN>(a, s))) return rc;
  a.A = (const float *)b.dab; a.am = 1; a.ak = 2 * f;            // dWgu = dab^T x
  a.B = (const float *)b.x; a.bn = 1; a.bk = d;
  a.M = 2 * b.f; a.N = b.d;
  a.C = (float *)b.dw_gate_up;
  return simt::launch<simt::PLAIN>(a, s);
}

}  // namespace ffn
}  // namespace moe
