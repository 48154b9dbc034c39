// The gated feed-forward block's forward for few tokens (up to 64), bf16: one token is the case of serving.
//
// Bound: the weights' way from HBM, 6 d f bytes, once. A thread block therefore owns a few output features (16 or 32 weight
// rows) over the whole of K, its eight warps an eighth of K each, and the weights go from memory to registers and from there into
// the products, without a stop in shared memory: nothing in a block uses a weight twice. The products are mma.m16n8k16
// (weights as the 16 rows, tokens as the 8 columns): at up to 64 tokens they take a fraction of the time of the loads,
// and unlike tcgen05 they read their operands from registers. K may be taken in any order as long as both operands take the
// same, so a lane loads 16 consecutive bytes of a weight row and of a token and feeds them to two products:
// lane 4 g + q holds row (token) g, k = 8 q .. 8 q + 7 of each 32. GATEUP's 16 rows are 8 gate rows and the same features' 8 up rows,
// so a lane's accumulators hold a and b of one feature. The warps' sums meet in shared memory, in a fixed order.
//
// Tokens are read through L2 by every block: with 32 weight rows per block half as often as with 16, which is worth it where
// tokens outnumber rows and there are blocks enough (few_fwd). DOWN starts as a dependent of GATEUP and loads its
// first weights while GATEUP runs.
#include "dependent.cuh"
#include "ffn.cuh"

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

// NT: groups of eight tokens. MT: groups of sixteen weight rows. CH: 32-deep steps whose loads are in flight together.
template <bool UP, int NT, int MT, int CH>
__global__ void __launch_bounds__(THREADS, 2) ffn_few_kernel(const Params p) {
  __shared__ float4 sums[WARPS][MT * NT][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
  const int steps = (p.K + 31) / 32, each = (steps + WARPS - 1) / WARPS;
  const int s0 = warp * each, s1 = min(steps, s0 + each);
  if (UP) start_next();
  // this lane's two weight rows of each group of sixteen
  const __nv_bfloat16 *rows[MT][2];
  bool have[MT][2];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int n = UP ? (blockIdx.x * MT + m) * 8 + g : (blockIdx.x * MT + m) * 16 + 8 * u + g;
      have[m][u] = n < p.N;
      rows[m][u] = p.w + ((int64_t)(UP ? u * p.N : 0) + n) * p.K + 8 * q;
    }
  }
  uint4 w[CH][MT][2];
  auto load_weights = [&](int s) {
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int k = (s + c) * 32;
#pragma unroll
      for (int m = 0; m < MT; ++m) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          w[c][m][u] = make_uint4(0, 0, 0, 0);
          if (s + c < s1 && k + 8 * q < p.K && have[m][u]) w[c][m][u] = weight16(rows[m][u] + k);
        }
      }
    }
  };
  load_weights(s0);
  wait_previous();
  float acc[MT][NT][4] = {};
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
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const uint4 a = w[c][m][0], b = w[c][m][1];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          mma16816(acc[m][n], a.x, b.x, a.y, b.y, x[c][n].x, x[c][n].y);
          mma16816(acc[m][n], a.z, b.z, a.w, b.w, x[c][n].z, x[c][n].w);
        }
      }
    }
  }
#pragma unroll
  for (int m = 0; m < MT; ++m) {
#pragma unroll
    for (int n = 0; n < NT; ++n) sums[warp][m * NT + n][lane] = make_float4(acc[m][n][0], acc[m][n][1], acc[m][n][2], acc[m][n][3]);
  }
  __syncthreads();
  for (int i = warp; i < MT * NT; i += WARPS) {
    float4 v = sums[0][i][lane];
#pragma unroll
    for (int s = 1; s < WARPS; ++s) {
      const float4 o = sums[s][i][lane];
      v.x += o.x;
      v.y += o.y;
      v.z += o.z;
      v.w += o.w;
    }
    const int m = i / NT, t = 8 * (i - m * NT) + 2 * q;   // tokens t and t + 1
    if (UP) {
      const int n = (blockIdx.x * MT + m) * 8 + g;
      if (n >= p.N) continue;
      if (t < p.T) p.out[(int64_t)t * p.N + n] = __float2bfloat16_rn(gated(v.x, p.gate) * v.z);
      if (t + 1 < p.T) p.out[(int64_t)(t + 1) * p.N + n] = __float2bfloat16_rn(gated(v.y, p.gate) * v.w);
    } else {
      const float r[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int n = (blockIdx.x * MT + m) * 16 + 8 * (e >> 1) + g, tt = t + (e & 1);
        if (n >= p.N || tt >= p.T) continue;
        const int64_t at = (int64_t)tt * p.N + n;
        p.out[at] = __float2bfloat16_rn(r[e] + (p.add ? __bfloat162float(p.add[at]) : 0.0f));
      }
    }
  }
}

template <bool UP, int NT, int MT, int CH> static int launch(const Params &p, cudaStream_t s) {
  const int per = UP ? 8 * MT : 16 * MT, grid = (p.N + per - 1) / per;
  if (UP) {
    ffn_few_kernel<UP, NT, MT, CH><<<grid, THREADS, 0, s>>>(p);
    MOE_CHECK_LAUNCH();
  } else {
    MOE_TRY_CUDA(launch_after(ffn_few_kernel<UP, NT, MT, CH>, dim3(grid), dim3(THREADS), 0, s, p));
  }
  return MOE_OK;
}
// 32 weight rows per block where more tokens than 16 read them and two blocks per SM remain.
template <bool UP> static int run(const Params &p, cudaStream_t s) {
  const int nt = (p.T + 7) / 8;
  const bool two = nt > 2 && (p.N + (UP ? 15 : 31)) / (UP ? 16 : 32) >= 2 * sm_count();
  if (nt == 1) return launch<UP, 1, 1, 8>(p, s);
  if (nt == 2) return launch<UP, 2, 1, 4>(p, s);
  if (nt <= 4) return two ? launch<UP, 4, 2, 2>(p, s) : launch<UP, 4, 1, 4>(p, s);
  return launch<UP, 8, 1, 2>(p, s);
}

}  // namespace few

int few_fwd(const Block &b, cudaStream_t s) {
  typedef __nv_bfloat16 bf16;
  few::Params p{};
  p.tok = (const bf16 *)b.x;
  p.w = (const bf16 *)b.w_gate_up;
  p.out = (bf16 *)b.h;
  p.T = b.T;
  p.K = b.d;
  p.N = b.f;
  p.gate = b.gate;
  const int rc = few::run<true>(p, s);
  if (rc) return rc;
  p.tok = (const bf16 *)b.h;
  p.w = (const bf16 *)b.w_down;
  p.add = (const bf16 *)b.add;
  p.out = (bf16 *)b.y;
  p.K = b.f;
  p.N = b.d;
  return few::run<false>(p, s);
}

}  // namespace ffn
}  // namespace moe
