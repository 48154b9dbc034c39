// Grouped expert FFN on MXFP4 operands for few rows per expert (decoding, small batches): the weights are the MMA's
// A operand and the tokens its N, so the tensor work follows the rows there are, and the bound is the weights'
// way from HBM. Same operands and results as the kernels in fp4_gemm.cu.
//
// One CTA computes 256 weight rows (two accumulators of 128 TMEM lanes) by up to 64 grouped rows (N, the routed
// rows rounded up to 16). GATEUP: the two are 128 gate rows and the same features' 128 up rows, so a lane of the
// epilogue holds a and b of one feature, a warp the 32 features of one MXFP4 block: its largest magnitude is one
// warp reduction per token, the codes go through shared memory to gather a token's 16 bytes in one lane. DOWN: a
// lane holds one output feature, a warp stores 64 consecutive bytes per token, rounded to bf16 (why: fp4_gemm.cu).
//
// With tokens as M (256 rows per pair, fp4_gemm.cu) a tile's MMAs take as long for one row as for 256. Measured (d = 2048,
// E = 64, k = 8, f = 1024), GATEUP reads its 142.6 MB of weights in 33-36 us at 42 rows per expert (4.0-4.3 TB/s with
// launch and last wave, 5.4 TB/s while all CTAs run); the ring's depth, the L2 promotion, the order of K and smaller
// tiles do not matter there.
//
// Two sets of accumulators (256 TMEM columns), scales behind them. A token tile that starts in the middle of a
// 128-row scale tile finds its scales two TMEM columns further. Roles, waits and dependent launch as in fp4_gemm.cu.
#include <atomic>

#include "fp4_gemm.cuh"

namespace moe {
namespace tc {
namespace fp4g {
namespace few {

constexpr int TT = 64;                                 // grouped rows per tile
constexpr int A_BYTES = 128 * 128, B_BYTES = TT * 128; // per stage: 128 weight rows, 64 token rows
constexpr int STAGE_BYTES = 2 * A_BYTES + B_BYTES + 3 * SF_BYTES;
constexpr int STAGES = 5;
constexpr int BUF_BYTES = 1024;                        // GATEUP: 32 tokens x 32 codes, one byte each, per warp
constexpr int NBARS = 2 * STAGES + 5;
constexpr uint32_t SET = 128;                          // columns of one set: two accumulators of 64
constexpr uint32_t SF_COL = 2 * SET, SF_SET = 24;      // scales: two sets of 8 + 8 (weights) + 8 (tokens) columns
static_assert(STAGE_BYTES % 1024 == 0, "ring stages keep the swizzle atoms' 1024-byte alignment");
template <int K> constexpr int smem_bytes() {
  return STAGES * STAGE_BYTES + (K == GATEUP ? EPI_WARPS * BUF_BYTES : 0) + 1024 + 8 * NBARS + 16 + (int)sizeof(Plan);
}
static_assert(smem_bytes<GATEUP>() <= 232448, "MXFP4 GEMM shared memory exceeds 227 KB");

__device__ __forceinline__ void arrive_here(uint32_t bar) {   // TMEM has been read (wait::ld); no memory is handed over
  asm volatile("mbarrier.arrive.relaxed.cta.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}
__device__ __forceinline__ uint32_t e2m1(float v) {           // one code, in the low four bits
  uint32_t r;
  asm("{\n\t.reg .b8 b;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %2, %1;\n\t"
      "cvt.u32.u8 %0, b;\n\t}"
      : "=r"(r)
      : "f"(v), "f"(0.0f));
  return r;
}

// f(c, this lane's value of token c in the first accumulator, in the second) for the `count` (warp-uniform) tokens from
// TMEM column `col` on. Eight at a time in a loop: unrolled over 32 tokens the code of a tile with one token is mostly
// jumped over, and fetching it cost 1 us per kernel.
template <typename F> __device__ __forceinline__ void for_tokens(uint32_t col, int count, F f) {
#pragma unroll 1
  for (int c0 = 0; c0 < count; c0 += 8) {
    uint32_t r0[8], r1[8];
    tmem_ld8(col + c0, r0);
    tmem_ld8(col + TT + c0, r1);
    tmem_ld_wait();
#pragma unroll
    for (int c = 0; c < 8; ++c)
      if (c0 + c < count) f(c0 + c, __uint_as_float(r0[c]), __uint_as_float(r1[c]));
  }
}

// tmT32: token codes, 32 rows per box; tmW: weight codes, 128 rows; tmST, tmSW: scales.
template <int K>
__global__ void __launch_bounds__(THREADS, 1)
    fp4_few_kernel(const __grid_constant__ CUtensorMap tmT32, const __grid_constant__ CUtensorMap tmW,
                   const __grid_constant__ CUtensorMap tmST, const __grid_constant__ CUtensorMap tmSW, const Params p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t *epi_smem = smem + STAGES * STAGE_BYTES;
  uint64_t *bars = reinterpret_cast<uint64_t *>(epi_smem + (K == GATEUP ? EPI_WARPS * BUF_BYTES : 0));
  // bars: full[STAGES], empty[STAGES], tfull[2], tempty[2], mma_done
  uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(bars + NBARS);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_holder + 1);
  Plan &plan = *reinterpret_cast<Plan *>(tmem_holder + 4);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t sbase = smem_u32(smem), bar0 = smem_u32(bars);
  auto full_bar = [&](int s) { return bar0 + 8u * s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (STAGES + s); };
  auto tfull_bar = [&](int a) { return bar0 + 8u * (2 * STAGES + a); };
  auto tempty_bar = [&](int a) { return bar0 + 8u * (2 * STAGES + 2 + a); };
  const uint32_t mma_done_bar = bar0 + 8u * (2 * STAGES + 4);

  // A tile's weights for `n` ring stages, into L2 (a hint)
  auto prefetch_weights = [&](const Tile &t, int n) {
    const int w0 = t.e * p.w_rows_e + t.ft * p.w_step, w1 = w0 + p.w_second;
    if (elect_one()) {
#pragma unroll 1
      for (int kb = 0; kb < n; ++kb) {
        prefetch_2d(&tmW, kb * 128, w0);
        prefetch_2d(&tmW, kb * 128, w1);
        prefetch_2d(&tmSW, kb * (SF_BYTES / 4), w0 / 128);
        prefetch_2d(&tmSW, kb * (SF_BYTES / 4), w1 / 128);
      }
    }
    __syncwarp();
  };

  if (K == DOWN) start_next();
  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(tfull_bar(a), 1);
      mbar_init(tempty_bar(a), EPI_WARPS);
    }
    mbar_init(mma_done_bar, 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    for (const CUtensorMap *m : {&tmW, &tmSW, &tmT32, &tmST})
      asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(m)) : "memory");
  }
  if (warp == 0) {   // see fp4_gemm.cu
    make_plan<TT>(p, lane, plan);
    if (K == GATEUP) {
      __syncwarp();
      Walker<TT> walk(blockIdx.x, gridDim.x, p, plan);
      Tile t;
      if (walk.next(t, p, plan)) prefetch_weights(t, min(p.num_kb, STAGES));
      __syncwarp();
      wait_previous();
      make_plan<TT, true>(p, lane, plan);
    }
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_holder)),
                 "r"(512u)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  if (K == GATEUP) start_next();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_holder;

  if (warp == 0) {
    // ------------------------------------------------------------------ producer
    int stage = 0, fills = 0;
    uint32_t phase = 0;
    bool ok = true;
    auto load_weights = [&](const Tile &t, int kb, int st) {
      const uint32_t sA = sbase + st * STAGE_BYTES, sS = sA + 2 * A_BYTES + B_BYTES, fb = full_bar(st);
      const int w0 = t.e * p.w_rows_e + t.ft * p.w_step, w1 = w0 + p.w_second;
      mbar_expect_tx(fb, 2 * A_BYTES + (uint32_t)((t.valid + 31) / 32) * (B_BYTES / 2) + 3 * SF_BYTES);
      tma_load_2d(sA, &tmW, kb * 128, w0, fb);
      tma_load_2d(sA + A_BYTES, &tmW, kb * 128, w1, fb);
      tma_load_2d(sS, &tmSW, kb * (SF_BYTES / 4), w0 / 128, fb);
      tma_load_2d(sS + SF_BYTES, &tmSW, kb * (SF_BYTES / 4), w1 / 128, fb);
    };
    auto load_tokens = [&](const Tile &t, int kb, int st) {
      const uint32_t sB = sbase + st * STAGE_BYTES + 2 * A_BYTES, fb = full_bar(st);
      for (int b = 0; 32 * b < t.valid; ++b) tma_load_2d(sB + b * (B_BYTES / 2), &tmT32, kb * 128, t.start + 32 * b, fb);
      tma_load_2d(sB + B_BYTES + 2 * SF_BYTES, &tmST, kb * (SF_BYTES / 4), t.start / 128, fb);
    };
    Walker<TT> walk(blockIdx.x, gridDim.x, p, plan);
    for (Tile t; ok && walk.next(t, p, plan);) {
      int kb = 0;
      if (fills == 0) {   // the first tile: the ring is empty. DOWN: the weights, then wait for GATEUP
        fills = kb = min(p.num_kb, STAGES);
        if (elect_one()) {
          for (int i = 0; i < kb; ++i) {
            load_weights(t, i, i);
            if (K == GATEUP) load_tokens(t, i, i);
          }
        }
        __syncwarp();
        if (K == DOWN) {
          // and the second tile's into L2, while GATEUP's last tiles leave HBM idle: 62.0 against 63.4 us for the FFN
          // at 333 tokens. (Every tile's successor, in both kernels: 69.7.)
          Walker<TT> ahead = walk;
          Tile u;
          if (ahead.next(u, p, plan)) prefetch_weights(u, p.num_kb);
          wait_previous();
          if (elect_one())
            for (int i = 0; i < kb; ++i) load_tokens(t, i, i);
          __syncwarp();
        }
        if (kb < STAGES) {
          stage = kb;
        } else {
          phase = 1;
        }
      }
      for (; kb < p.num_kb; ++kb) {
        if (!mbar_spin_cluster(empty_bar(stage), phase ^ 1u, abort_flag, p.hdr, 51)) { ok = false; break; }
        if (elect_one()) {
          load_weights(t, kb, stage);
          load_tokens(t, kb, stage);
        }
        __syncwarp();
        ++fills;
        if (++stage == STAGES) { stage = 0; phase ^= 1u; }
      }
    }
    if (K == DOWN && fills == 0) wait_previous();
    if (*abort_flag) {   // leave no copy in flight: wait (bounded) for the last fill of every stage
      const uint64_t t0 = global_ns();
      for (int i = 1; i <= STAGES && i <= fills; ++i) {
        const int f = fills - i;   // fill number f went to stage f % STAGES in ring round f / STAGES
        while (!mbar_try_wait(full_bar(f % STAGES), (uint32_t)(f / STAGES) & 1u) && global_ns() - t0 < kWaitLimitNs) {}
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------------ MMA issuer
    wait_previous();
    int stage = 0, acc = 0, set = 0;
    uint32_t phase = 0, acc_phase = 0;
    bool issued = false, ok = true;
    const uint64_t desc_a0 = sdesc(sbase, 16, 1024), desc_b0 = sdesc(sbase + 2 * A_BYTES, 16, 1024);
    const uint64_t desc_s0 = sf_desc(sbase + 2 * A_BYTES + B_BYTES);
    Walker<TT> walk(blockIdx.x, gridDim.x, p, plan);
    for (Tile t; ok && walk.next(t, p, plan);) {
      if (!mbar_spin_cluster(tempty_bar(acc), acc_phase ^ 1u, abort_flag, p.hdr, 52)) break;
      tc_fence_after();
      const uint32_t d0 = tmem_base + (uint32_t)acc * SET, d1 = d0 + TT;
      const int n = (t.valid + 15) & ~15;
      const uint32_t half = (uint32_t)(t.start >> 6) & 1u;   // which half of its 128-row scale tile
      for (int kb = 0; kb < p.num_kb; ++kb) {
        if (!mbar_spin_cluster(full_bar(stage), phase, abort_flag, p.hdr, 53)) { ok = false; break; }
        tc_fence_after();
        if (elect_one()) {
          const uint32_t so = (uint32_t)(stage * STAGE_BYTES) >> 4;
          const uint32_t sf = tmem_base + SF_COL + (uint32_t)set * SF_SET;   // weights 0, weights 1, tokens: 8 columns each
#pragma unroll
          for (int h = 0; h < 2; ++h) {   // 128 values of K each
#pragma unroll
            for (int o = 0; o < 3; ++o)
              copy_scales<1>(sf + 8 * o + 4 * h, desc_s0 + so + (uint32_t)((o * SF_BYTES + h * 512) >> 4));
#pragma unroll
            for (int kk = 0; kk < 2; ++kk) {
              const uint32_t koff = (uint32_t)((2 * h + kk) * 32) >> 4, id = idesc(128, n, 2u * kk);
              const uint32_t go = (kb | h | kk) != 0 ? 1u : 0u, sft = sf + 16 + 4 * h + 2 * half;
              mma_mxf4<1>(d0, desc_a0 + so + koff, desc_b0 + so + koff, id, sf + 4 * h, sft, go);
              mma_mxf4<1>(d1, desc_a0 + so + (A_BYTES >> 4) + koff, desc_b0 + so + koff, id, sf + 8 + 4 * h, sft, go);
            }
          }
          mma_commit(empty_bar(stage));
        }
        __syncwarp();
        issued = true;
        set ^= 1;
        if (++stage == STAGES) { stage = 0; phase ^= 1u; }
      }
      if (!ok) break;
      if (elect_one()) mma_commit(tfull_bar(acc));
      __syncwarp();
      acc ^= 1;
      if (acc == 0) acc_phase ^= 1u;
    }
    if (issued) {   // every MMA is done before TMEM is freed
      if (elect_one()) mma_commit(mma_done_bar);
      __syncwarp();
      const uint64_t t0 = global_ns();
      while (!mbar_try_wait(mma_done_bar, 0) && global_ns() - t0 < kWaitLimitNs) {}
    }
  } else {
    // ------------------------------------------------------------------ epilogue
    wait_previous();
    const int quarter = warp & 3, hh = (warp - 2) >> 2;   // this warp's 32 lanes; its tokens 32 hh .. 32 hh + 31
    const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
    const uint32_t buf = smem_u32(epi_smem) + (uint32_t)(warp - 2) * BUF_BYTES;
    int acc = 0;
    uint32_t acc_phase = 0;
    Walker<TT> walk(blockIdx.x, gridDim.x, p, plan);
    for (Tile t; walk.next(t, p, plan);) {
      if (!mbar_spin_cluster(tfull_bar(acc), acc_phase, abort_flag, p.hdr, 54)) break;
      tc_fence_after();
      const uint32_t tacc = tmem_base + lane_off + (uint32_t)acc * SET + 32u * hh;
      const int cnt = min(32, max(0, t.valid - 32 * hh));
      auto drained = [&] {   // this warp has read its part of the accumulators
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_here(tempty_bar(acc));
        acc ^= 1;
        if (acc == 0) acc_phase ^= 1u;
      };
      const int64_t row0 = (int64_t)t.start + 32 * hh;
      // the rows to write: the expert's last tile writes its padding's zeros
      const int64_t pad = ((int64_t)t.start + t.valid + 127) / 128 * 128;
      const int64_t end = !t.last ? (int64_t)t.start + TT : (pad < p.rows_max ? pad : p.rows_max);
      if (K == GATEUP) {
        uint32_t mine = 0;                    // lane c: scale byte of token c
        for_tokens(tacc, cnt, [&](int c, float a, float b) {
          const float h = a * b * sigmoidf_(a);
          const uint32_t byte = fp4::scale_byte(__reduce_max_sync(0xffffffffu, __float_as_uint(h) & 0x7fffffffu));
          const uint32_t code = byte == 255u ? 0u : e2m1(h * fp4::inv_scale(byte));
          asm volatile("st.shared.u8 [%0], %1;" ::"r"(buf + 32u * c + lane), "r"(code) : "memory");
          if (lane == c) mine = byte;
        });
        drained();
        uint4 q = make_uint4(0, 0, 0, 0);     // lane c: the 32 codes of token c
        if (lane < cnt) {
          const uint4 lo = ld_shared_v4(buf + 32u * lane), hi = ld_shared_v4(buf + 32u * lane + 16u);
          auto two = [](uint32_t a, uint32_t b) { return __byte_perm(a | a >> 4, b | b >> 4, 0x6420); };
          q = make_uint4(two(lo.x, lo.y), two(lo.z, lo.w), two(hi.x, hi.y), two(hi.z, hi.w));
        }
        __syncwarp();                         // the buffer is read before the next tile writes it
        for (int64_t row = row0 + lane; row < end; row += TT) {   // further rows: padding
          *reinterpret_cast<uint4 *>(p.h + row * (p.f / 2) + t.ft * 64 + 16 * quarter) = q;
          p.h_scales[fp4::scale_word(row, t.ft, p.f / 128) + quarter] = (uint8_t)mine;
          q = make_uint4(0, 0, 0, 0);
          mine = 0;
        }
      } else {
        __nv_bfloat16 *y = p.y + row0 * p.d + t.ft * 256 + 32 * quarter;
        for_tokens(tacc, cnt, [&](int c, float v0, float v1) {
          y[(int64_t)c * p.d + lane] = __float2bfloat16_rn(v0);
          y[(int64_t)c * p.d + 128 + lane] = __float2bfloat16_rn(v1);
        });
        drained();
        // zeros in the rows past the routed ones: four lanes per 64 bytes of a row
        for (int64_t base = row0; base < end; base += TT) {
          for (int i = base == row0 ? cnt : 0; i < 32; i += 8) {
            const int rr = i + (lane >> 2);
            if (rr < 32 && base + rr < end) {
              uint4 *dst = reinterpret_cast<uint4 *>(p.y + (base + rr) * p.d + t.ft * 256 + 32 * quarter) + (lane & 3);
              dst[0] = make_uint4(0, 0, 0, 0);
              dst[16] = make_uint4(0, 0, 0, 0);   // 128 features on
            }
          }
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(512u) : "memory");
  }
}

template <int K> static int launch(const Maps &m, const Params &p, cudaStream_t s) {
  static std::atomic<uint64_t> raised{0};   // devices on which the kernel's shared memory limit has been raised
  int dev = 0;
  MOE_TRY_CUDA(cudaGetDevice(&dev));
  if (dev >= 64 || !(raised.load(std::memory_order_relaxed) >> dev & 1)) {
    MOE_TRY_CUDA(cudaFuncSetAttribute(fp4_few_kernel<K>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes<K>()));
    if (dev < 64) raised.fetch_or((uint64_t)1 << dev, std::memory_order_relaxed);
  }
  int64_t grid = sm_count();
  const int64_t most = p.rows_max / TT * p.n_ft;   // tiles there can be
  if (most < grid) grid = most;
  MOE_TRY_CUDA(launch_after(fp4_few_kernel<K>, dim3((unsigned)grid), dim3(THREADS), smem_bytes<K>(), s, m.a32, m.b, m.sa,
                            m.sb, p));
  return MOE_OK;
}

}  // namespace few

int few_gateup(const Maps &m, const Params &p, cudaStream_t s) { return few::launch<GATEUP>(m, p, s); }
int few_down(const Maps &m, const Params &p, cudaStream_t s) { return few::launch<DOWN>(m, p, s); }

}  // namespace fp4g
}  // namespace tc
}  // namespace moe
