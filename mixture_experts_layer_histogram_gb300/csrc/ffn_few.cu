// The gated feed-forward block's forward for few tokens (up to 64), bf16: one token is the case of serving.
//
// Bound: the weights' way from HBM, 6 d f bytes, once. A thread block therefore owns a few output features (16 weight rows) over
// the whole of K, its eight warps an eighth of K each, and the weights go from memory to registers and from there into the
// products, without a stop in shared memory: nothing in a block uses a weight twice. The products are mma.m16n8k16 (weights as
// the 16 rows, tokens as the 8 columns): at up to 64 tokens they take a fraction of the time of the loads, and unlike tcgen05
// they read their operands from registers. K may be taken in any order as long as both operands take the same, so a lane loads
// 16 consecutive bytes of a weight row and of a token and feeds them to two products: lane 4 g + q holds row (token) g, k = 8 q
// .. 8 q + 7 of each 32. GATEUP's 16 rows are 8 gate rows and the same features' 8 up rows, so a lane's accumulators hold a and
// b of one feature. The warps' sums meet in shared memory, in a fixed order.
//
// DOWN starts as a dependent of GATEUP and loads its first weights while GATEUP runs.
// Measured at 2048 x 1024 (12.6 MB of weights, in L2): one token 4.3 us in a replayed graph, 8.1 us in a stream of calls (the
// host's time); 16 tokens 5.8 us. Both products in one cooperative launch, with a count of finished blocks between them, took
// 5.3 and 7.3 us in a graph and saved 1.6 us of host time.
#include <cuda.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "dependent.cuh"
#include "ffn.cuh"
#include "stages.h"
#include "tc_ptx.cuh"
#include "tma_host.cuh"

namespace moe {
namespace ffn {
namespace few {

constexpr int WARPS = 8;
constexpr int THREADS = 32 * WARPS;

struct Params {
  const __nv_bfloat16 *tok;    // [T, K]: x or h
  const __nv_bfloat16 *w;      // rows of K values
  const __nv_bfloat16 *add;    // DOWN (null: nothing)
  __nv_bfloat16 *out;          // GATEUP h [T, N], DOWN y [T, N]
  int T, K, N;                 // N: f or d
  Gate gate;
};

// A weight's 16 bytes, read once: past L1. (Through the coherent path: DOWN runs beside GATEUP, see dependent.cuh.)
__device__ __forceinline__ uint4 weight16(const __nv_bfloat16 *p) { return ld_stream_coherent(reinterpret_cast<const uint4 *>(p)); }

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// A lane's four sums: a (v.x, v.y) and b (v.z, v.w) of feature n for tokens t and t + 1 ...
__device__ __forceinline__ void put_up(const Params &p, int n, int t, const float4 &v) {
  if (n >= p.N) return;
  if (t < p.T) p.out[(int64_t)t * p.N + n] = __float2bfloat16_rn(gated(v.x, p.gate) * v.z);
  if (t + 1 < p.T) p.out[(int64_t)(t + 1) * p.N + n] = __float2bfloat16_rn(gated(v.y, p.gate) * v.w);
}
// ... or y of columns n and n + apart for tokens t and t + 1
__device__ __forceinline__ void put_down(const Params &p, int n, int apart, int t, const float4 &v) {
  const float r[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int nn = n + apart * (e >> 1), tt = t + (e & 1);
    if (nn >= p.N || tt >= p.T) continue;
    const int64_t at = (int64_t)tt * p.N + nn;
    p.out[at] = __float2bfloat16_rn(r[e] + (p.add ? __bfloat162float(p.add[at]) : 0.0f));
  }
}

// NT: groups of eight tokens. CH: 32-deep steps whose loads are in flight together.
template <bool UP, int NT, int CH>
__global__ void __launch_bounds__(THREADS, 2) ffn_few_kernel(const Params p) {
  __shared__ float4 sums[WARPS][NT][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
  const int steps = (p.K + 31) / 32, each = (steps + WARPS - 1) / WARPS;
  const int s0 = warp * each, s1 = min(steps, s0 + each);
  if (UP) start_next();
  // this lane's two weight rows
  const __nv_bfloat16 *rows[2];
  bool have[2];
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int n = UP ? blockIdx.x * 8 + g : blockIdx.x * 16 + 8 * u + g;
    have[u] = n < p.N;
    rows[u] = p.w + ((int64_t)(UP ? u * p.N : 0) + n) * p.K + 8 * q;
  }
  uint4 w[CH][2];
  auto load_weights = [&](int s) {
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int k = (s + c) * 32;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        w[c][u] = make_uint4(0, 0, 0, 0);
        if (s + c < s1 && k + 8 * q < p.K && have[u]) w[c][u] = weight16(rows[u] + k);
      }
    }
  };
  load_weights(s0);
  wait_previous();
  float acc[NT][4] = {};
  for (int s = s0; s < s1; s += CH) {
    if (s > s0) load_weights(s);
    uint4 x[CH][NT];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int k = (s + c) * 32 + 8 * q;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        x[c][n] = make_uint4(0, 0, 0, 0);
        if (s + c < s1 && k < p.K && 8 * n + g < p.T)
          x[c][n] = *reinterpret_cast<const uint4 *>(p.tok + (int64_t)(8 * n + g) * p.K + k);
      }
    }
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const uint4 a = w[c][0], b = w[c][1];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        mma16816(acc[n], a.x, b.x, a.y, b.y, x[c][n].x, x[c][n].y);
        mma16816(acc[n], a.z, b.z, a.w, b.w, x[c][n].z, x[c][n].w);
      }
    }
  }
#pragma unroll
  for (int n = 0; n < NT; ++n) sums[warp][n][lane] = make_float4(acc[n][0], acc[n][1], acc[n][2], acc[n][3]);
  __syncthreads();
  for (int i = warp; i < NT; i += WARPS) {
    float4 v = sums[0][i][lane];
#pragma unroll
    for (int s = 1; s < WARPS; ++s) {
      const float4 o = sums[s][i][lane];
      v.x += o.x;
      v.y += o.y;
      v.z += o.z;
      v.w += o.w;
    }
    const int t = 8 * i + 2 * q;   // tokens t and t + 1
    if (UP) put_up(p, blockIdx.x * 8 + g, t, v);
    else put_down(p, blockIdx.x * 16 + g, 8, t, v);
  }
}

template <bool UP, int NT, int CH> static int launch(const Params &p, cudaStream_t s) {
  constexpr int per = UP ? 8 : 16;
  const int grid = (p.N + per - 1) / per;
  if (UP) {
    ffn_few_kernel<UP, NT, CH><<<grid, THREADS, 0, s>>>(p);
    MOE_CHECK_LAUNCH();
  } else {
    MOE_TRY_CUDA(launch_after(ffn_few_kernel<UP, NT, CH>, dim3(grid), dim3(THREADS), 0, s, p));
  }
  return MOE_OK;
}

// ---------------------------------------------------------------------------------------------
// The same for weights that keep the GPU busy for longer than a kernel takes to start: one block per SM streams its row groups
// through a ring in shared memory that TMA keeps full, 16 (or 32) weight rows and all tokens by 512 of K a stage, whatever the
// registers hold; each of the eight warps takes 64 of the 512. The tensors are seen as [K / 64, rows, 64], so that one copy
// brings eight 128-byte-swizzled boxes: 16-byte chunk c of row g lies at (c ^ g) * 16 (g its low three bits). A lane takes the
// chunks 2 q and 2 q + 1, so that the eight lanes that read together, of two rows, meet all banks once (q and q + 4 met half of
// them twice). Measured for 24 tokens of 4096 x 8192: 26.5 us for the 134 MB of Wg and Wu (5.1 TB/s) and 16 for the 67 MB of Wd,
// 41 together; with loads into registers (above) the 134 MB took 33 us.
constexpr int KS = 512;                        // of K per stage
constexpr int BOX = 8 * KS * 2;                // bytes of 8 rows of a stage
struct Stream {
  // Units of 16 weight rows (8 gate and the same features' 8 up rows, or 16 of Wd); a group takes MT of them, or (mixed) MT while
  // groups are below `full`, then one
  int full, groups, steps;                     // steps: stages per group
};
// Groups of two kinds, for up to 16 tokens; their units come in boxes of 8 rows then, else in one box per half. (Small boxes
// cost 3% with 24 tokens, where the shorter last round gains nothing.)
template <int NT, int MT> constexpr bool mixed() { return NT <= 2 && MT == 2; }
template <int NT, int MT> constexpr int weight_bytes() { return 2 * MT * BOX; }
template <int NT> constexpr int token_bytes() { return NT * BOX; }
template <int NT, int MT> constexpr int stage_bytes() { return weight_bytes<NT, MT>() + token_bytes<NT>(); }
template <int NT, int MT> constexpr int sum_bytes() { return WARPS * MT * NT * 512; }
constexpr int kSmemMost = 232448;
template <int NT, int MT> constexpr int stages_with(int sums) {
  const int n = (kSmemMost - 2048 - sums * sum_bytes<NT, MT>()) / stage_bytes<NT, MT>();
  return n > 8 ? 8 : n;
}
template <int NT, int MT> constexpr int stages_of() { return stages_with<NT, MT>(1); }
// The warps' sums in two buffers in turn, one barrier a group, where that costs no stage; else in one, with two barriers
template <int NT, int MT> constexpr int sums_of() { return stages_with<NT, MT>(2) == stages_of<NT, MT>() ? 2 : 1; }
template <int NT, int MT> constexpr int smem_of() {
  return stages_of<NT, MT>() * stage_bytes<NT, MT>() + sums_of<NT, MT>() * sum_bytes<NT, MT>() + 1024 + 256;
}

__device__ __forceinline__ void load_3d(uint32_t dst, const CUtensorMap *map, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}

// tmW: boxes of 8 weight rows (8 MT unless mixed), tmX: boxes of 8 NT tokens, each 64 x 8 of K
template <bool UP, int NT, int MT>
__global__ void __launch_bounds__(THREADS + 32, 1)
    ffn_stream_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX, const Params p, const Stream st,
                      WsHeader *hdr) {
  constexpr int PS = stages_of<NT, MT>(), SB = stage_bytes<NT, MT>(), SUMS = sums_of<NT, MT>();
  constexpr bool MIXED = mixed<NT, MT>();
  constexpr int ROWS = MIXED ? 8 : 8 * MT;     // of a box
  extern __shared__ uint8_t raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  float4(*sums)[MT * NT][32] = reinterpret_cast<float4(*)[MT * NT][32]>(smem + PS * SB);
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + PS * SB + SUMS * sum_bytes<NT, MT>());   // full[PS], empty[PS]
  volatile int *abort_flag = reinterpret_cast<volatile int *>(bars + 2 * PS);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
  const uint32_t base = tc::smem_u32(smem), bar0 = tc::smem_u32(bars);
  auto full = [&](int s) { return bar0 + 8u * s; };
  auto empty = [&](int s) { return bar0 + 8u * (PS + s); };
  if (UP) start_next();
  if (threadIdx.x == 0) {
    for (int s = 0; s < PS; ++s) {
      tc::mbar_init(full(s), 1);
      tc::mbar_init(empty(s), WARPS);
    }
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncthreads();
  const int mine = (int)blockIdx.x < st.groups ? (st.groups - 1 - (int)blockIdx.x) / (int)gridDim.x + 1 : 0;
  const int total = mine * st.steps;           // stages that this block goes through
  auto whole = [&](int gr) { return !MIXED || gr < st.full; };
  auto first = [&](int gr) { return whole(gr) ? gr * MT : gr + st.full * (MT - 1); };   // the group's first unit
  if (warp == WARPS) {
    // ---- the ring's producer: one elected lane
    if (tc::elect_one()) {
      auto weights = [&](int i) {
        const int gr = (int)blockIdx.x + i / st.steps * (int)gridDim.x, k = i % st.steps, s = i % PS;
        const bool all = whole(gr);
        tc::mbar_expect_tx(full(s), (all ? MT : 1) * 2 * BOX + token_bytes<NT>());
        for (int m = 0; m < (MIXED && all ? MT : 1); ++m) {
          const int row = (first(gr) + m) * (UP ? 8 : 16);
          load_3d(base + s * SB + m * BOX, &tmW, 0, row, k * (KS / 64), full(s));
          load_3d(base + s * SB + (MT + m) * BOX, &tmW, 0, UP ? p.N + row : row + ROWS, k * (KS / 64), full(s));
        }
      };
      auto tokens = [&](int i) {
        const int k = i % st.steps, s = i % PS;
        load_3d(base + s * SB + weight_bytes<NT, MT>(), &tmX, 0, 0, k * (KS / 64), full(s));
      };
      const int head = total < PS ? total : PS;
      for (int i = 0; i < head; ++i) weights(i);   // the weights do not wait for the kernel before
      wait_previous();
      for (int i = 0; i < head; ++i) tokens(i);
      for (int i = head; i < total; ++i) {
        if (!tc::mbar_wait(empty(i % PS), (uint32_t)(i / PS - 1) & 1u, abort_flag, hdr, 51)) break;
        weights(i);
        tokens(i);
      }
    }
  } else {
    wait_previous();
    float acc[MT][NT][4] = {};
    int gr = blockIdx.x, at_sums = 0;
    auto there = [&](int i) {   // lanes look one by one, but the warp goes on, or gives up, together
      const uint32_t phase = (uint32_t)(i / PS) & 1u;
      const bool seen = tc::mbar_try_wait(full(i % PS), phase) || tc::mbar_wait(full(i % PS), phase, abort_flag, hdr, 52);
      return __all_sync(0xffffffffu, seen) != 0;
    };
    auto use = [&](int i) {
      const int s = i % PS;
      const uint32_t w0 = base + s * SB + (uint32_t)warp * (ROWS * 128), x0 = base + s * SB + weight_bytes<NT, MT>() + (uint32_t)warp * (NT * 1024);
      auto products = [&](auto count) {   // of the group's units
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t at = (uint32_t)g * 128 + (((uint32_t)(2 * q + h) ^ (uint32_t)g) << 4);
          uint4 x[NT];
#pragma unroll
          for (int n = 0; n < NT; ++n) x[n] = tc::ld_shared_v4(x0 + n * 1024 + at);
#pragma unroll
          for (int m = 0; m < decltype(count)::value; ++m) {
            const uint32_t w = w0 + m * (MIXED ? BOX : 1024) + at;
            const uint4 a = tc::ld_shared_v4(w), b = tc::ld_shared_v4(w + MT * BOX);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              mma16816(acc[m][n], a.x, b.x, a.y, b.y, x[n].x, x[n].y);
              mma16816(acc[m][n], a.z, b.z, a.w, b.w, x[n].z, x[n].w);
            }
          }
        }
      };
      if (whole(gr)) products(std::integral_constant<int, MT>());
      else products(std::integral_constant<int, 1>());
      // the reads above come before the TMA's next writes to this place: another proxy's, which the arrival alone does not order
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(empty(s));
    };
    // the group's sums over the warps, in their order (of an unfinished group nothing is written by a warp that knows)
    auto meet = [&](bool ok) {
#pragma unroll
      for (int m = 0; m < MT; ++m) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          sums[at_sums + warp][m * NT + n][lane] = make_float4(acc[m][n][0], acc[m][n][1], acc[m][n][2], acc[m][n][3]);
          acc[m][n][0] = acc[m][n][1] = acc[m][n][2] = acc[m][n][3] = 0.0f;
        }
      }
      asm volatile("bar.sync 1, %0;" ::"n"(THREADS) : "memory");
      for (int j = warp; ok && j < (whole(gr) ? MT : 1) * NT; j += WARPS) {
        float4 v = sums[at_sums][j][lane];
#pragma unroll
        for (int u = 1; u < WARPS; ++u) {
          const float4 o = sums[at_sums + u][j][lane];
          v.x += o.x;
          v.y += o.y;
          v.z += o.z;
          v.w += o.w;
        }
        const int m = j / NT, t = 8 * (j - m * NT) + 2 * q;   // tokens t and t + 1
        if (UP) put_up(p, 8 * (first(gr) + m) + g, t, v);
        else put_down(p, 16 * first(gr) + (MIXED ? 16 : 8) * m + g, ROWS, t, v);
      }
      if (SUMS == 1) asm volatile("bar.sync 1, %0;" ::"n"(THREADS) : "memory");
      else at_sums ^= WARPS;
      gr += gridDim.x;
    };
    const bool ok = through_stages(total, st.steps, there, use, meet);
    if (!ok) {   // copies in flight land within microseconds
      const uint64_t t0 = global_ns();
      while (global_ns() - t0 < 1000ull * 1000ull) {}
    }
  }
}

// [rows, K] bf16 seen as [K / 64, rows, 64], boxes of 64 x box_rows x 8
static bool stream_map(CUtensorMap *m, const void *p, uint64_t rows, uint64_t K, uint32_t box_rows) {
  tc::EncodeTiledFn enc = tc::encode_fn();
  if (!enc) return false;
  cuuint64_t dims[3] = {64, rows, K / 64}, strides[2] = {K * 2, 128};
  cuuint32_t box[3] = {64, box_rows, KS / 64}, one[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(p), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
template <auto KERNEL, int SMEM> static int raise_limit() {
  static std::atomic<uint64_t> raised{0};
  int dev = 0;
  MOE_TRY_CUDA(cudaGetDevice(&dev));
  if (dev < 64 && (raised.load(std::memory_order_relaxed) >> dev & 1)) return MOE_OK;
  MOE_TRY_CUDA(cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM));
  if (dev < 64) raised.fetch_or((uint64_t)1 << dev, std::memory_order_relaxed);
  return MOE_OK;
}
template <bool UP, int NT, int MT> static int launch_stream(const Params &p, int full, int groups, WsHeader *hdr, cudaStream_t s) {
  constexpr int SMEM = smem_of<NT, MT>();
  static_assert(SMEM <= kSmemMost && stages_of<NT, MT>() >= 2, "two stages at least");
  CUtensorMap mw, mx;
  if (!stream_map(&mw, p.w, UP ? 2 * (uint64_t)p.N : p.N, p.K, mixed<NT, MT>() ? 8 : 8 * MT) || !stream_map(&mx, p.tok, p.T, p.K, 8 * NT)) return MOE_ERR_CUDA;
  const int rc = raise_limit<ffn_stream_kernel<UP, NT, MT>, SMEM>();
  if (rc) return rc;
  const Stream st{full, groups, (p.K + KS - 1) / KS};
  const int grid = std::min(groups, sm_count());
  if (UP) {
    ffn_stream_kernel<UP, NT, MT><<<grid, THREADS + 32, SMEM, s>>>(mw, mx, p, st, hdr);
    MOE_CHECK_LAUNCH();
  } else {
    MOE_TRY_CUDA(launch_after(ffn_stream_kernel<UP, NT, MT>, dim3(grid), dim3(THREADS + 32), (size_t)SMEM, s, mw, mx, p, st, hdr));
  }
  return MOE_OK;
}
template <bool UP, int NT> static int stream(const Params &p, WsHeader *hdr, cudaStream_t s) {
  const int units = (p.N + (UP ? 7 : 15)) / (UP ? 8 : 16), sms = sm_count();
  if constexpr (NT <= 2) {
    // Groups of two units, which read the tokens half as often, while they fill rounds over the SMs; what is left in single units
    // where that is one round, half as long: 17.3 against 20.5 us for one token of 2048 x 8192.
    int full = units / (2 * sms) * sms, rest = units - 2 * full;
    if (rest > sms) {
      full += rest / 2;
      rest &= 1;
    }
    if (full > 0) return launch_stream<UP, NT, 2>(p, full, full + rest, hdr, s);
  } else if constexpr (NT <= 4) {
    // Groups of two where they take no longer in whole rounds than single units, of which more stages fit.
    const int pairs = (units + 1) / 2;
    if (2 * ((pairs + sms - 1) / sms) <= (units + sms - 1) / sms) return launch_stream<UP, NT, 2>(p, pairs, pairs, hdr, s);
  }
  return launch_stream<UP, NT, 1>(p, 0, units, hdr, s);
}

// ring: through the ring, both products of a call
template <bool UP> static int run(const Params &p, bool ring, WsHeader *hdr, cudaStream_t s) {
  const int nt = (p.T + 7) / 8;
  if (ring) {
    switch (nt) {
      case 1: return stream<UP, 1>(p, hdr, s);
      case 2: return stream<UP, 2>(p, hdr, s);
      case 3: return stream<UP, 3>(p, hdr, s);
      case 4: return stream<UP, 4>(p, hdr, s);
      case 5:
      case 6: return stream<UP, 6>(p, hdr, s);
      default: return stream<UP, 8>(p, hdr, s);
    }
  }
  if (nt == 1) return launch<UP, 1, 8>(p, s);
  if (nt == 2) return launch<UP, 2, 4>(p, s);
  if (nt <= 4) return launch<UP, 4, 4>(p, s);
  return launch<UP, 8, 2>(p, s);
}

}  // namespace few

// Small weights take the kernel that starts quickest, others the ring, whose rows are whole 128 bytes. In us, the ring and the
// other: 4 tokens of 2048 x 1024 (12.6 MB) 8.9 and 8.0, of 2048 x 2048 10.1 and 8.2, of 4096 x 2048 (50 MB) 12.3 and 12.3, of
// 2048 x 8192 (101 MB) 20 and 25; 24 tokens of 768 x 512 (2.4 MB) 8.7 and 7.9, of 2048 x 1024 8.9 and 9.0, of 2048 x 2048 10.3
// and 12.3. (One product through the ring and the other not is slower than either: 14.1 for 4 tokens of 4096 x 2048.)
bool few_ring(int T, int d, int f) {
  return d % 64 == 0 && f % 64 == 0 && (int64_t)6 * d * f > (int64_t)(T <= 16 ? 48 : 8) << 20;
}

int few_fwd(const Block &b, cudaStream_t s) {
  typedef __nv_bfloat16 bf16;
  const bool ring = few_ring(b.T, b.d, b.f);
  few::Params p{};
  p.tok = (const bf16 *)b.x;
  p.w = (const bf16 *)b.w_gate_up;
  p.out = (bf16 *)b.h;
  p.T = b.T;
  p.K = b.d;
  p.N = b.f;
  p.gate = b.gate;
  const int rc = few::run<true>(p, ring, b.hdr, s);
  if (rc) return rc;
  p.tok = (const bf16 *)b.h;
  p.w = (const bf16 *)b.w_down;
  p.add = (const bf16 *)b.add;
  p.out = (bf16 *)b.y;
  p.K = b.f;
  p.N = b.d;
  return few::run<false>(p, ring, b.hdr, s);
}

}  // namespace ffn
}  // namespace moe
