// What the grouped MXFP4 products share: parameters, descriptors and tensor maps.
#pragma once

#include <cuda.h>

#include "common.cuh"
#include "dependent.cuh"
#include "fp4.cuh"
#include "tc_ptx.cuh"
#include "tma_host.cuh"

namespace moe {
namespace tc {
namespace fp4g {

enum Kind { GATEUP = 0, DOWN = 1 };

constexpr int KS = 256;                       // values of K per ring stage (128 bytes of codes: the swizzle span)
constexpr int SF_BYTES = (KS / 128) * 512;    // scales of 128 rows per stage
constexpr int EPI_WARPS = 8;
constexpr int THREADS = 64 + 32 * EPI_WARPS;
constexpr int MAX_E = MOE_MAX_EXPERTS;

struct Params {
  const int32_t *tile_offsets, *offsets;
  WsHeader *hdr;
  int E;
  int n_ft;               // feature tiles per expert
  int num_kb;             // ring stages per tile
  int w_rows_e;           // weight rows per expert
  int w_second;           // rows from a tile's first 128 weight rows to its second (GATEUP: f, DOWN: 128)
  int w_step;             // weight rows from one feature tile to the next
  uint8_t *h, *h_scales;  // GATEUP
  __nv_bfloat16 *y;       // DOWN
  int d, f;
  int64_t rows_max;
};

// Instruction descriptor, kind::mxf4: A and B E2M1, scales E8M0, both K-major; sf = the first of the two scale bytes (0
// or 2) of each operand.
__device__ __forceinline__ uint32_t idesc(int m, int n, uint32_t sf) {
  return (sf << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) | (1u << 23) | ((uint32_t)(m >> 4) << 24) |
         (sf << 29);
}
template <int CTAS>
__device__ __forceinline__ void mma_mxf4(uint32_t d, uint64_t ad, uint64_t bd, uint32_t id, uint32_t sfa, uint32_t sfb,
                                         uint32_t accumulate) {
  if (CTAS == 2)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
        "l"(ad), "l"(bd), "r"(id), "r"(sfa), "r"(sfb), "r"(accumulate));
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
        "l"(ad), "l"(bd), "r"(id), "r"(sfa), "r"(sfb), "r"(accumulate));
}
// 512 bytes of scales (32 rows of 16 bytes) to four TMEM columns, repeated in each 32-lane quarter; of a pair,
// each CTA from its own shared memory to its own TMEM.
template <int CTAS> __device__ __forceinline__ void copy_scales(uint32_t taddr, uint64_t desc) {
  if (CTAS == 2) asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc));
  else asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc));
}
// Shared-memory descriptor without swizzle: core matrices of 8 rows x 16 bytes, 128 bytes apart.
__device__ __forceinline__ uint64_t sf_desc(uint32_t saddr) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(128 >> 4) << 32) | (1ull << 46);
}

// 2D codes [rows, bytes per row], boxes of 128 bytes x box_rows rows, 128-byte swizzle.
inline bool codes_map(CUtensorMap *m, const void *base, uint64_t rows, uint64_t row_bytes, uint32_t box_rows) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  cuuint64_t dims[2] = {row_bytes, rows};
  cuuint64_t strides[1] = {row_bytes};
  cuuint32_t box[2] = {128, box_rows};
  cuuint32_t estr[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Scales of [rows, K] (rows, K multiples of 128) as 32-bit words [rows / 128, K]: a box is the 1024 bytes of one stage.
inline bool scales_map(CUtensorMap *m, const void *base, uint64_t rows, uint64_t k) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  cuuint64_t dims[2] = {k, rows / 128};
  cuuint64_t strides[1] = {k * 4};
  cuuint32_t box[2] = {SF_BYTES / 4, 1};
  cuuint32_t estr[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, const_cast<void *>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Fetch a box into L2 (a hint: nothing depends on what it reads or when).
__device__ __forceinline__ void prefetch_2d(const CUtensorMap *m, int x, int y) {
  asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(reinterpret_cast<uint64_t>(m)),
               "r"(x), "r"(y)
               : "memory");
}

// The experts' rows, as tiles of TR, in shared memory.
struct Plan {
  int tiles[MAX_E + 1];      // token tiles before expert e
  int first[MAX_E];          // its first grouped row / 128
  uint16_t last[MAX_E];      // routed rows in its last tile (1..TR)
};
// Filled by one warp. The offsets are read from L2: the kernel may have started, and read them, before the kernel
// that writes them had ended. An expert whose rows do not lie inside its row group, or whose group does not lie inside
// the buffers, counts as empty (REPORT: and MOE_ERR_CHECK_FAILED is recorded): every row that a tile touches is below rows_max.
template <int TR, bool REPORT = false> __device__ __forceinline__ void make_plan(const Params &p, int lane, Plan &plan) {
  int c[8], at[9], o[9], sum = 0;
#pragma unroll
  for (int q = 0; q < 9; ++q) {
    const int e = min(lane * 8 + q, p.E);
    o[q] = __ldcg(p.offsets + e);
    at[q] = __ldcg(p.tile_offsets + e);
  }
#pragma unroll
  for (int q = 0; q < 8; ++q) c[q] = o[q + 1] - o[q];
  const uint32_t groups = (uint32_t)(p.rows_max / MOE_GROUP_ROWS);
  auto fits = [&](int q) {   // unsigned: what is negative is too large
    const uint32_t first = (uint32_t)at[q], next = (uint32_t)at[q + 1];
    return first <= next && next <= groups && (uint32_t)c[q] <= (next - first) * MOE_GROUP_ROWS;
  };
  bool fit = true;
#pragma unroll
  for (int q = 0; q < 8; ++q) fit = fit && fits(q);
  if (!fit) {
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      if (fits(q)) continue;
      c[q] = 0;
      if (REPORT) report(p.hdr, MOE_ERR_CHECK_FAILED, min(lane * 8 + q, p.E - 1));
    }
  }
#pragma unroll
  for (int q = 0; q < 8; ++q) sum += (c[q] + TR - 1) / TR;
  int incl = sum;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, off);
    if (lane >= off) incl += v;
  }
  int run = incl - sum;
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    const int e = lane * 8 + q, n = (c[q] + TR - 1) / TR;
    if (e < p.E) {
      plan.tiles[e] = run;
      plan.first[e] = at[q];
      plan.last[e] = (uint16_t)(c[q] - (n - 1) * TR);
    }
    run += n;
  }
  if (lane == 31) plan.tiles[p.E] = incl;
}

struct Tile {
  int e, ft, start, valid;   // expert, feature tile, first grouped row, routed rows (1..TR)
  bool last;                 // the expert's last rows
};
// One CTA's (or pair's) tiles in order: first, first + step, ...; tile = token tile * n_ft + feature tile. A whole warp calls
// next(): one expert after the other, the search for the first tile's took 3.4 us at E = 64. Whatever the plan
// holds, e < E and ft < n_ft.
template <int TR> struct Walker {
  int tile, step, num, e;
  __device__ __forceinline__ Walker(int first, int step_, const Params &p, const Plan &plan)
      : tile(first), step(step_), num(plan.tiles[p.E] * p.n_ft), e(0) {}
  __device__ __forceinline__ bool next(Tile &t, const Params &p, const Plan &plan) {
    if (tile >= num) return false;
    const int gt = tile / p.n_ft;
    t.ft = tile - gt * p.n_ft;
    const int lane = threadIdx.x & 31;
    for (;;) {   // 32 experts at a time
      const int i = e + 1 + lane, n = __popc(__ballot_sync(0xffffffffu, i < p.E && plan.tiles[min(i, p.E)] <= gt));
      e += n;
      if (n < 32) break;
    }
    const int i = gt - plan.tiles[e];
    t.e = e;
    t.start = plan.first[e] * 128 + i * TR;
    t.last = gt + 1 == plan.tiles[e + 1];
    t.valid = t.last ? plan.last[e] : TR;
    tile += step;
    return true;
  }
};

struct Maps {
  CUtensorMap a, a32, b, sa, sb, c;   // token codes in boxes of 128 and of 32 rows, weight codes, scales, y (DOWN)
};
// The products for few rows per expert (fp4_gemm_few.cu).
int few_gateup(const Maps &m, const Params &p, cudaStream_t s);
int few_down(const Maps &m, const Params &p, cudaStream_t s);

}  // namespace fp4g
}  // namespace tc
}  // namespace moe
