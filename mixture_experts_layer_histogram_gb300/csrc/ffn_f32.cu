// The gated feed-forward block in true fp32 (FFMA on the CUDA cores; tf32 tensor cores would not hold fp32), any sizes.
//
// One kernel for the five products: C[m, n] = sum_k A(m, k) B(n, k), operands addressed by strides (K-major and MN-major
// alike). 16-deep steps through a ring in shared memory, filled element by element with cp.async (rows of odd length
// start anywhere), three steps ahead; two fp32 per instruction from 8 x 8 values per thread (a tile of 128 x 128) or 8 x 4
// (64 x 64, where 128 would leave SMs idle). GATEUP takes gate rows for the first half of a tile's columns and the same
// features' up rows for the second. The finished tile passes through shared memory, from where neighbouring threads write
// neighbouring columns.
//
// A product with few tiles and a long K is shared by up to eight blocks of a cluster, a part of K each: each block leaves its
// tile in its shared memory and finishes a share of the rows, adding the parts up in the blocks' order. Products that do not
// wait for one another share a launch (dh with dWd, dx with dWgu), the one of longer blocks first: its end is filled by the
// other. Measured at 203 x 501 x 1337 (2.4 GFLOP), forward and backward: 409 us without the cluster and with one step in flight,
// 155 with both, 137 with addresses formed once and K cut by the work per SM, 113 with four launches instead of six and
// addresses as steps from the first (fewer registers); at 2000 x 1024 x 2048 (75 GFLOP) 1.67 ms, 45 TFLOP/s. What is left in the
// small case: the ramps of four launches, SMs that get three blocks where others get two, and rows and columns past the edge
// (203 rows are computed as 256). Tried and not kept: the kernels as dependents of one another (145 against 127 us then), 8 x 8
// values per thread in the small tile with two groups of threads that share its K (115-119 us), steps of 32 (156), three blocks
// per SM with more registers (123).
#include <cooperative_groups.h>

#include <algorithm>
#include <atomic>

#include "f32x2.cuh"
#include "ffn.cuh"

namespace moe {
namespace ffn {
namespace simt {

namespace cg = cooperative_groups;

enum Kind { GATEUP = 0, PLAIN = 1, DH = 2 };

constexpr int BK = 16, STAGES = 4, MAX_SPLIT = 8;

// One product
struct Args {
  int kind, cols, tiles;     // tile columns, and tiles in all
  int splits;                // blocks that share a tile, a part of K each: a power of two, at most the cluster's size
  const float *A, *B;
  int64_t am, ak, bn, bk;    // strides
  int M, N, K;               // N: columns of the result (GATEUP, DH: f)
  float *C;                  // GATEUP kept ab (null: not kept); DH dab; PLAIN the result
  float *C2;                 // GATEUP h
  const float *in;           // DH kept ab; PLAIN what is added (null: nothing)
  Gate gate;
};
// One launch: a product, or two that do not wait for one another; the second one's blocks follow the first one's (whole clusters)
struct Job {
  Args p[2];
  int blocks0;
};

template <int B> struct Tile;   // B x B outputs, TM x TN per thread; BLOCKS: per SM
template <> struct Tile<64> { static constexpr int TM = 8, TN = 4, THREADS = 128, BLOCKS = 4; };
template <> struct Tile<128> { static constexpr int TM = 8, TN = 8, THREADS = 256, BLOCKS = 2; };
template <int B> constexpr int ld() { return B + 4; }                                   // floats per k row of an operand
template <int B> constexpr int stage_floats() { return 2 * BK * ld<B>(); }
template <int B> constexpr int smem_bytes() { return STAGES * stage_floats<B>() * 4; }   // the finished tile fits in it
static_assert(smem_bytes<64>() >= 64 * 66 * 4 && smem_bytes<128>() >= 128 * 130 * 4, "the tile takes the ring's place");

__device__ __forceinline__ void copy4(uint32_t dst, const float *src, bool there) {   // zero where there is nothing
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(there ? 4 : 0) : "memory");
}

// A product's blocks: tile * splits + part, tiles row by row
template <int B> __global__ void __launch_bounds__(Tile<B>::THREADS, Tile<B>::BLOCKS) ffn_f32_kernel(const __grid_constant__ Job job) {
  using S = Tile<B>;
  constexpr int TM = S::TM, TN = S::TN, THREADS = S::THREADS, LD = ld<B>(), PER = B * BK / THREADS, TX = B / TN;
  constexpr int HALF = B / 2, GM = TM / 2, GN = TN / 2;   // a thread's rows and columns lie in both halves of the tile
  extern __shared__ __align__(16) float ring[];
  cg::cluster_group cluster = cg::this_cluster();
  const int second = (int)blockIdx.x >= job.blocks0 ? 1 : 0;
  const Args p = second ? job.p[1] : job.p[0];   // (job.p[second] would be read through a generic address, each time)
  const bool gate_up = p.kind == GATEUP;
  const int id = (int)blockIdx.x - (second ? job.blocks0 : 0), splits = p.splits, tile = id / splits, part = id - tile * splits;
  if (tile >= p.tiles) {             // the cluster's last blocks may have nothing to do
    cluster.sync();
    cluster.sync();
    return;
  }
  const int tx = threadIdx.x % TX, ty = threadIdx.x / TX;
  const int m0 = tile / p.cols * B, n0 = tile % p.cols * (gate_up ? HALF : B);
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
  const int ra0 = a_k ? threadIdx.x / BK : threadIdx.x % B, rb0 = b_k ? threadIdx.x / BK : threadIdx.x % B;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int ra = a_k ? ra0 + i * RK : ra0, rb = b_k ? rb0 + i * RK : rb0;
    if (m0 + ra < p.M) a_rows |= 1u << i;
    if (n0 + (gate_up && rb >= HALF ? rb - HALF : rb) < p.N) b_rows |= 1u << i;
  }
  pa += (int64_t)(m0 + ra0) * p.am;
  pb += (int64_t)(n0 + rb0) * p.bn;
  const int64_t a_step = a_k ? RK * p.am : RM * p.ak, b_step = b_k ? RK * p.bn : RM * p.bk;
  const int64_t b_jump = gate_up ? (int64_t)(p.N - HALF) * p.bn : 0;   // from gate rows to up rows (K-major)
  static_assert(RK * (PER / 2) == HALF, "the second half of a thread's rows lies in the tile's second half");
  const uint32_t a_dst = (uint32_t)(ka0 * LD + ra0) * 4, b_dst = (uint32_t)(kb0 * LD + rb0) * 4 + BK * LD * 4;
  const uint32_t a_dst_step = a_k ? RK * 4 : RM * LD * 4, b_dst_step = b_k ? RK * 4 : RM * LD * 4;
  int left = p.K - s0 * BK;          // of K from the next step to fetch on
  auto fetch = [&](int s) {
    if (s < s1) {
      const uint32_t at = base + (uint32_t)(s % STAGES) * (stage_floats<B>() * 4);
      const float *qa = pa, *qb = pb;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const bool ok = (a_rows >> i & 1) && (a_k ? ka0 : ka0 + i * RM) < left;
        copy4(at + a_dst + i * a_dst_step, ok ? qa : p.A, ok);
        qa += a_step;
        if (i == PER / 2) qb += b_jump;
        const bool okb = (b_rows >> i & 1) && (b_k ? kb0 : kb0 + i * RM) < left;
        copy4(at + b_dst + i * b_dst_step, okb ? qb : p.B, okb);
        qb += b_step;
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
  cluster.sync();
  // this block's share of the rows; a thread per column
  const int columns = gate_up ? HALF : B, rows = THREADS / columns, c = threadIdx.x % columns, r1 = B * (part + 1) / splits;
  const int rank0 = (int)cluster.block_rank() - part;
  auto sum = [&](int at) {
    if (splits == 1) return ring[at];
    float w[MAX_SPLIT], v = 0.0f;
#pragma unroll
    for (int q = 0; q < MAX_SPLIT; ++q) w[q] = q < splits ? cluster.map_shared_rank(ring, rank0 + q)[at] : 0.0f;   // all on their way at once
#pragma unroll
    for (int q = 0; q < MAX_SPLIT; ++q) v += w[q];
    return v;
  };
  const int64_t n = n0 + c;
#pragma unroll 2
  for (int r = B * part / splits + threadIdx.x / columns; r < r1; r += rows) {
    const int64_t m = m0 + r;
    if (m >= p.M || n >= p.N) continue;
    const float v = sum(r * LT + c);
    if (gate_up) {
      const float b = sum(r * LT + HALF + c);
      if (p.C) {
        p.C[m * 2 * p.N + n] = v;
        p.C[m * 2 * p.N + p.N + n] = b;
      }
      p.C2[m * p.N + n] = gated<true>(v, p.gate) * b;
    } else if (p.kind == DH) {
      const float a = p.in[m * 2 * p.N + n], b = p.in[m * 2 * p.N + p.N + n];
      float act, slope;
      gate_and_slope(a, p.gate, act, slope);
      p.C[m * 2 * p.N + n] = v * b * slope;
      p.C[m * 2 * p.N + p.N + n] = v * act;
    } else {
      p.C[m * p.N + n] = v + (p.in ? p.in[m * p.N + n] : 0.0f);
    }
  }
  cluster.sync();                    // no block leaves while another reads its tile
}

static int64_t up(int64_t n, int64_t k) { return (n + k - 1) / k; }
static int64_t tiles_of(const Args &a, int B) { return up(a.M, B) * up((a.kind == GATEUP ? 2 : 1) * (int64_t)a.N, B); }

template <int B> static int launch_tile(Job &job, int n, int size, cudaStream_t s) {
  int64_t blocks[2] = {0, 0};
  for (int i = 0; i < n; ++i) {
    Args &a = job.p[i];
    const int64_t tiles = tiles_of(a, B);
    blocks[i] = up(tiles * a.splits, size) * size;
    if (blocks[i] > 0x3fffffff) return MOE_ERR_UNSUPPORTED;
    a.cols = (int)up((a.kind == GATEUP ? 2 : 1) * (int64_t)a.N, B);
    a.tiles = (int)tiles;
  }
  job.blocks0 = (int)blocks[0];
  static std::atomic<uint64_t> raised{0};   // once per device: the limit is the process's
  int dev = 0;
  MOE_TRY_CUDA(cudaGetDevice(&dev));
  if (dev >= 64 || !(raised.load(std::memory_order_relaxed) >> dev & 1)) {
    MOE_TRY_CUDA(cudaFuncSetAttribute(ffn_f32_kernel<B>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes<B>()));
    if (dev < 64) raised.fetch_or((uint64_t)1 << dev, std::memory_order_relaxed);
  }
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = (unsigned)size;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(blocks[0] + blocks[1]));
  cfg.blockDim = dim3(Tile<B>::THREADS);
  cfg.dynamicSmemBytes = smem_bytes<B>();
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  MOE_TRY_CUDA(cudaLaunchKernelEx(&cfg, ffn_f32_kernel<B>, job));
  return MOE_OK;
}

// One or two products in a launch. Tiles of 128 where they fill the GPU twice over, else of 64, with K cut into the numbers of
// parts that give the shortest time: the work per SM and half a longest block for the uneven end, but no less than two of those
// (a block that has an SM to itself, four warps, takes about twice as long per step as those that share it). A block counts its
// steps and four more for its start and end. Longer blocks start first.
static int launch(Args *a, int n, cudaStream_t s) {
  const int64_t sms = sm_count();
  Job job{};
  if (tiles_of(a[0], 128) + (n > 1 ? tiles_of(a[1], 128) : 0) >= 2 * sms) {
    const int first = n > 1 && a[1].K > a[0].K;
    for (int i = 0; i < n; ++i) {
      job.p[i] = a[first ^ i];
      job.p[i].splits = 1;
    }
    return launch_tile<128>(job, n, 1, s);
  }
  int64_t least = INT64_MAX;
  int best[2] = {1, 1};
  auto length = [&](int i, int splits) { return up(up(a[i].K, BK), splits) + 4; };
  for (int x = 1; x <= MAX_SPLIT; x *= 2) {
    for (int y = 1; y <= (n > 1 ? MAX_SPLIT : 1); y *= 2) {
      int64_t work = tiles_of(a[0], 64) * x * length(0, x), longest = length(0, x);
      if (n > 1) {
        work += tiles_of(a[1], 64) * y * length(1, y);
        longest = std::max(longest, length(1, y));
      }
      const int64_t cost = std::max(2 * longest, work / sms + longest / 2);
      if (cost < least) {
        least = cost;
        best[0] = x;
        best[1] = y;
      }
    }
  }
  const int first = n > 1 && length(1, best[1]) > length(0, best[0]);
  for (int i = 0; i < n; ++i) {
    job.p[i] = a[first ^ i];
    job.p[i].splits = best[first ^ i];
  }
  return launch_tile<64>(job, n, std::max(best[0], best[1]), s);
}

}  // namespace simt

using simt::Args;

int f32_fwd(const Block &b, cudaStream_t s) {
  Args a{};
  a.kind = simt::GATEUP;
  a.A = (const float *)b.x; a.am = b.d; a.ak = 1;
  a.B = (const float *)b.w_gate_up; a.bn = b.d; a.bk = 1;
  a.M = b.T; a.N = b.f; a.K = b.d;
  a.C = (float *)b.ab; a.C2 = (float *)b.h;
  a.gate = b.gate;
  const int rc = simt::launch(&a, 1, s);
  if (rc) return rc;
  a.kind = simt::PLAIN;
  a.A = (const float *)b.h; a.am = b.f;
  a.B = (const float *)b.w_down; a.bn = b.f;
  a.N = b.d; a.K = b.f;
  a.C = (float *)b.y; a.in = (const float *)b.add;
  return simt::launch(&a, 1, s);
}

int f32_bwd(const Block &b, cudaStream_t s) {
  const int64_t f = b.f, d = b.d;
  Args a[2]{};
  a[0].kind = simt::DH;                                                // dh = dy Wd
  a[0].gate = b.gate;
  a[0].A = (const float *)b.dy; a[0].am = d; a[0].ak = 1;
  a[0].B = (const float *)b.w_down; a[0].bn = 1; a[0].bk = f;
  a[0].M = b.T; a[0].N = b.f; a[0].K = b.d;
  a[0].in = (const float *)b.ab; a[0].C = (float *)b.dab;
  a[1].kind = simt::PLAIN;                                             // dWd = dy^T h
  a[1].A = (const float *)b.dy; a[1].am = 1; a[1].ak = d;
  a[1].B = (const float *)b.h; a[1].bn = 1; a[1].bk = f;
  a[1].M = b.d; a[1].N = b.f; a[1].K = b.T;
  a[1].C = (float *)b.dw_down;
  const int rc = simt::launch(a, 2, s);
  if (rc) return rc;
  a[0].kind = simt::PLAIN;                                             // dx = dab Wgu
  a[0].A = (const float *)b.dab; a[0].am = 2 * f; a[0].ak = 1;
  a[0].B = (const float *)b.w_gate_up; a[0].bn = 1; a[0].bk = d;
  a[0].N = b.d; a[0].K = 2 * b.f;
  a[0].in = (const float *)b.add; a[0].C = (float *)b.dx;
  a[1].A = (const float *)b.dab; a[1].am = 1; a[1].ak = 2 * f;         // dWgu = dab^T x
  a[1].B = (const float *)b.x; a[1].bn = 1; a[1].bk = d;
  a[1].M = 2 * b.f; a[1].N = b.d;
  a[1].C = (float *)b.dw_gate_up;
  return simt::launch(a, 2, s);
}

}  // namespace ffn
}  // namespace moe
