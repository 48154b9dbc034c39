// The gated feed-forward block in true fp32 (FFMA on the CUDA cores; tf32 tensor cores would not hold fp32), any sizes.
//
// One kernel for the five products: C[m, n] = sum_k A(m, k) B(n, k), operands addressed by strides (K-major and MN-major
// alike). 16-deep steps through a ring in shared memory, filled element by element with cp.async (rows of odd length
// start anywhere), three steps ahead; two fp32 per instruction from 8 x 8 values per thread (a tile of 128 x 128) or 8 x 4
// (64 x 64, where 128 would leave SMs idle). GATEUP takes gate rows for the first half of a tile's columns and the same
// features' up rows for the second. The finished tile passes through shared memory, from where neighbouring threads write
// neighbouring columns.
//
// A product with few tiles and a long K is shared by a cluster of up to eight blocks, a part of K each: each block leaves its
// tile in its shared memory and finishes a share of the rows, adding the parts up in the blocks' order. Measured at 203 x 501 x
// 1337 (2.4 GFLOP), forward and backward: 409 us without the cluster and with one step in flight, 155 with both, 130 in a
// replayed graph (140 in a stream of calls) with addresses formed once and K cut by the work per SM; at 2000 x 1024 x 2048 (75
// GFLOP) 1.81 ms, 42 TFLOP/s. There the FMA pipe is active 69% of the time and waits for its turn; the small case keeps it 44%
// active: SMs that get three blocks where others get two, the ramp of six launches, and rows and columns past the edge (203 rows
// are computed as 256). Launched as dependents of one another the six kernels took 145 us; 8 x 8 values per thread in the small
// tile, two groups of threads sharing its K, took the same time.
#include <cooperative_groups.h>

#include <atomic>

#include "f32x2.cuh"
#include "ffn.cuh"

namespace moe {
namespace ffn {
namespace simt {

namespace cg = cooperative_groups;

enum Kind { GATEUP = 0, PLAIN = 1, DH = 2 };

constexpr int BK = 16, STAGES = 4, MAX_SPLIT = 8;

struct Args {
  const float *A, *B;
  int64_t am, ak, bn, bk;    // strides
  int M, N, K;               // N: columns of the result (GATEUP, DH: f)
  float *C;                  // GATEUP kept ab (null: not kept); DH dab; PLAIN the result
  float *C2;                 // GATEUP h
  const float *in;           // DH kept ab; PLAIN what is added (null: nothing)
  Gate gate;
};

template <int B> struct Tile;   // B x B outputs, TM x TN per thread
template <> struct Tile<64> { static constexpr int TM = 8, TN = 4, THREADS = 128; };
template <> struct Tile<128> { static constexpr int TM = 8, TN = 8, THREADS = 256; };
template <int B> constexpr int ld() { return B + 4; }                                   // floats per k row of an operand
template <int B> constexpr int stage_floats() { return 2 * BK * ld<B>(); }
template <int B> constexpr int smem_bytes() { return STAGES * stage_floats<B>() * 4; }   // the finished tile fits in it
static_assert(smem_bytes<64>() >= 64 * 66 * 4 && smem_bytes<128>() >= 128 * 130 * 4, "the tile takes the ring's place");

__device__ __forceinline__ void copy4(uint32_t dst, const float *src, bool there) {   // zero where there is nothing
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(there ? 4 : 0) : "memory");
}

// blockIdx.x = (tile column) * splits + part, splits = the cluster's size; blockIdx.y = tile row
template <int KIND, int B> __global__ void __launch_bounds__(Tile<B>::THREADS) ffn_f32_kernel(const Args p) {
  using S = Tile<B>;
  constexpr int TM = S::TM, TN = S::TN, THREADS = S::THREADS, LD = ld<B>(), PER = B * BK / THREADS, TX = B / TN;
  constexpr int HALF = B / 2, GM = TM / 2, GN = TN / 2;   // a thread's rows and columns lie in both halves of the tile
  extern __shared__ __align__(16) float ring[];
  cg::cluster_group cluster = cg::this_cluster();
  const int splits = (int)cluster.num_blocks(), part = (int)cluster.block_rank();
  const int tx = threadIdx.x % TX, ty = threadIdx.x / TX;
  const int m0 = blockIdx.y * B, n0 = (blockIdx.x / splits) * (KIND == GATEUP ? HALF : B);
  const int all = (p.K + BK - 1) / BK;
  const int s0 = (int)((int64_t)all * part / splits), s1 = (int)((int64_t)all * (part + 1) / splits);
  const uint32_t base = (uint32_t)__cvta_generic_to_shared(ring);
  // Element i of this thread: consecutive threads along the axis whose stride is 1. Its place and address are formed once; a
  // step moves all of them by BK along k.
  const bool a_k = p.ak == 1, b_k = p.bk == 1;
  const int ka0 = a_k ? threadIdx.x % BK : threadIdx.x / B, kb0 = b_k ? threadIdx.x % BK : threadIdx.x / B;
  constexpr int RK = THREADS / BK, RM = THREADS / B > 0 ? THREADS / B : 1;   // rows (along k) or k (along rows) between elements
  static_assert(THREADS % B == 0, "a thread keeps its row where threads run along rows");
  const float *pa = p.A + (int64_t)(s0 * BK + ka0) * p.ak, *pb = p.B + (int64_t)(s0 * BK + kb0) * p.bk;
  uint32_t a_rows = 0, b_rows = 0;   // which rows exist
  int64_t a_off[PER], b_off[PER];
  uint32_t a_dst[PER], b_dst[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int ra = a_k ? threadIdx.x / BK + i * RK : threadIdx.x % B, rb = b_k ? threadIdx.x / BK + i * RK : threadIdx.x % B;
    int64_t row = n0 + rb;
    bool ok = row < p.N;
    if (KIND == GATEUP && rb >= HALF) {
      ok = n0 + rb - HALF < p.N;
      row = (int64_t)p.N + n0 + rb - HALF;
    }
    if (m0 + ra < p.M) a_rows |= 1u << i;
    if (ok) b_rows |= 1u << i;
    a_off[i] = (int64_t)(m0 + ra) * p.am + (a_k ? 0 : i * RM * p.ak);
    b_off[i] = row * p.bn + (b_k ? 0 : i * RM * p.bk);
    a_dst[i] = (uint32_t)((a_k ? ka0 : ka0 + i * RM) * LD + ra) * 4;
    b_dst[i] = (uint32_t)((b_k ? kb0 : kb0 + i * RM) * LD + rb) * 4 + BK * LD * 4;
  }
  int left = p.K - s0 * BK;          // of K from the next step to fetch on
  auto fetch = [&](int s) {
    if (s < s1) {
      const uint32_t at = base + (uint32_t)(s % STAGES) * (stage_floats<B>() * 4);
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const bool ok = (a_rows >> i & 1) && (a_k ? ka0 : ka0 + i * RM) < left;
        copy4(at + a_dst[i], ok ? pa + a_off[i] : p.A, ok);
        const bool okb = (b_rows >> i & 1) && (b_k ? kb0 : kb0 + i * RM) < left;
        copy4(at + b_dst[i], okb ? pb + b_off[i] : p.B, okb);
      }
      pa += BK * p.ak;
      pb += BK * p.bk;
      left -= BK;
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  F2 acc[TM][TN / 2];
#pragma unroll
  for (int i = 0; i < TM; ++i) {
#pragma unroll
    for (int j = 0; j < TN / 2; ++j) acc[i][j] = pair(0.0f, 0.0f);
  }
  for (int s = 0; s < STAGES - 1; ++s) fetch(s0 + s);
  for (int s = s0; s < s1; ++s) {
    asm volatile("cp.async.wait_group %0;" ::"n"(STAGES - 2) : "memory");
    __syncthreads();                 // everyone's copies of this step are there, and everyone has left the step before,
    fetch(s + STAGES - 1);           // whose place is filled again
    const float *as = ring + (s % STAGES) * stage_floats<B>(), *bs = as + BK * LD;
#pragma unroll
    for (int k = 0; k < BK; ++k) {
      float a[TM];
      F2 b[TN / 2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float4 q = *reinterpret_cast<const float4 *>(as + k * LD + h * HALF + ty * GM);
        a[h * GM] = q.x;
        a[h * GM + 1] = q.y;
        a[h * GM + 2] = q.z;
        a[h * GM + 3] = q.w;
#pragma unroll
        for (int j = 0; j < GN / 2; ++j)
          b[h * (GN / 2) + j].v = *reinterpret_cast<const uint64_t *>(bs + k * LD + h * HALF + tx * GN + 2 * j);
      }
#pragma unroll
      for (int i = 0; i < TM; ++i) {
        const F2 aa = pair(a[i], a[i]);
#pragma unroll
        for (int j = 0; j < TN / 2; ++j) acc[i][j] = fma(aa, b[j], acc[i][j]);
      }
    }
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  __syncthreads();
  constexpr int LT = B + 2;          // floats per row of the finished tile
#pragma unroll
  for (int i = 0; i < TM; ++i) {
    const int r = (i / GM) * HALF + ty * GM + i % GM;
#pragma unroll
    for (int j = 0; j < TN / 2; ++j)
      *reinterpret_cast<uint64_t *>(ring + r * LT + (2 * j / GN) * HALF + tx * GN + 2 * j % GN) = acc[i][j].v;
  }
  if (splits > 1) cluster.sync();
  else __syncthreads();
  // this block's share of the rows; a thread per column
  constexpr int COLS = KIND == GATEUP ? HALF : B, ROWS = THREADS / COLS;
  const int c = threadIdx.x % COLS, r1 = B * (part + 1) / splits;
  auto sum = [&](int at) {
    if (splits == 1) return ring[at];
    float v = 0.0f;
    for (int q = 0; q < splits; ++q) v += cluster.map_shared_rank(ring, q)[at];
    return v;
  };
  const int64_t n = n0 + c;
  for (int r = B * part / splits + threadIdx.x / COLS; r < r1; r += ROWS) {
    const int64_t m = m0 + r;
    if (m >= p.M || n >= p.N) continue;
    const float v = sum(r * LT + c);
    if (KIND == GATEUP) {
      const float b = sum(r * LT + HALF + c);
      if (p.C) {
        p.C[m * 2 * p.N + n] = v;
        p.C[m * 2 * p.N + p.N + n] = b;
      }
      p.C2[m * p.N + n] = gated<true>(v, p.gate) * b;
    } else if (KIND == DH) {
      const float a = p.in[m * 2 * p.N + n], b = p.in[m * 2 * p.N + p.N + n];
      float act, slope;
      gate_and_slope(a, p.gate, act, slope);
      p.C[m * 2 * p.N + n] = v * b * slope;
      p.C[m * 2 * p.N + p.N + n] = v * act;
    } else {
      p.C[m * p.N + n] = v + (p.in ? p.in[m * p.N + n] : 0.0f);
    }
  }
  if (splits > 1) cluster.sync();    // no block leaves while another reads its tile
}

template <int KIND, int B> static int launch_tile(const Args &a, int64_t cols, int64_t rows, int splits, cudaStream_t s) {
  if (rows > 65535 || cols * splits > 0x7fffffff) return MOE_ERR_UNSUPPORTED;
  static std::atomic<uint64_t> raised{0};   // once per device: the limit is the process's
  int dev = 0;
  MOE_TRY_CUDA(cudaGetDevice(&dev));
  if (dev >= 64 || !(raised.load(std::memory_order_relaxed) >> dev & 1)) {
    MOE_TRY_CUDA(cudaFuncSetAttribute(ffn_f32_kernel<KIND, B>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes<B>()));
    if (dev < 64) raised.fetch_or((uint64_t)1 << dev, std::memory_order_relaxed);
  }
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = (unsigned)splits;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(cols * splits), (unsigned)rows);
  cfg.blockDim = dim3(Tile<B>::THREADS);
  cfg.dynamicSmemBytes = smem_bytes<B>();
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  MOE_TRY_CUDA(cudaLaunchKernelEx(&cfg, ffn_f32_kernel<KIND, B>, a));
  return MOE_OK;
}

// Tiles of 128 where they fill the GPU twice over, else of 64, with K cut into the number of parts (powers of two) that gives the
// shortest work per SM: the most blocks that one gets, times a part's steps and about four more for its start and end. Blocks
// that have an SM to themselves (four warps) take about twice as long per step as those that share it.
template <int KIND> static int launch(const Args &a, cudaStream_t s) {
  auto up = [](int64_t n, int64_t k) { return (n + k - 1) / k; };
  const int64_t sms = sm_count(), wide = KIND == GATEUP ? 2 : 1;
  if (up(a.M, 128) * up(wide * a.N, 128) >= 2 * sms) return launch_tile<KIND, 128>(a, up(wide * a.N, 128), up(a.M, 128), 1, s);
  const int64_t cols = up(wide * a.N, 64), rows = up(a.M, 64), steps = up(a.K, BK);
  int splits = 1;
  int64_t least = INT64_MAX;
  for (int n = 1; n <= MAX_SPLIT && n <= steps; n *= 2) {
    const int64_t per_sm = up(rows * cols * n, sms), cost = (per_sm < 2 ? 2 : per_sm) * (up(steps, n) + 4);
    if (cost < least) {
      least = cost;
      splits = n;
    }
  }
  return launch_tile<KIND, 64>(a, cols, rows, splits, s);
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
