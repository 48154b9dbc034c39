// What the grouped MXFP4 products share: parameters, descriptors and tensor maps.
#pragma once

#include <cuda.h>

#include "common.cuh"
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

// Exclusive scan of the token tiles per expert, ceil(rows / tile_rows), into shared memory: ttoff[0..E]. One warp.
__device__ __forceinline__ void scan_tiles(const Params &p, int tile_rows, int lane, int *ttoff) {
  int c[8], sum = 0;
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    const int e = lane * 8 + q;
    c[q] = e < p.E ? (p.offsets[e + 1] - p.offsets[e] + tile_rows - 1) / tile_rows : 0;
    sum += c[q];
  }
  int incl = sum;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, off);
    if (lane >= off) incl += v;
  }
  int run = incl - sum;
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    const int e = lane * 8 + q;
    if (e < p.E) ttoff[e] = run;
    run += c[q];
  }
  if (lane == 31) ttoff[p.E] = incl;
}

struct Maps {
  CUtensorMap a, a32, b, sa, sb, c;   // token codes in boxes of 128 and of 32 rows, weight codes, scales, y (DOWN)
};
// The products for few rows per expert (fp4_gemm_few.cu).
int few_gateup(const Maps &m, const Params &p, cudaStream_t s);
int few_down(const Maps &m, const Params &p, cudaStream_t s);

}  // namespace fp4g
}  // namespace tc
}  // namespace moe
