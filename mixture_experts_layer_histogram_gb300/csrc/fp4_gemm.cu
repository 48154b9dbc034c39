// Grouped expert FFN on MXFP4 operands: block-scaled tensor cores (sm_103a, tcgen05.mma kind::mxf4),
// forward only.
//
//   GATEUP  [a | b] = xq Wgu[e]^T, h = silu(a) b, written as MXFP4 (codes and scales)
//   DOWN    y = hq Wd[e]^T, written as bf16
//
// y is rounded to bf16, once per routed row, before the combine adds a token's k rows in fp32 and rounds again: the
// output is off by 2.4e-3 of its norm against 1.7e-3 with fp32 rows (d = 2048, k = 8; the codes of h and the products are
// the same in both). The rows are the combine's, as in the bf16 layer; in fp32 they would be twice the bytes, 268 MB more
// written here and read there at 8192 tokens: the combine alone takes 99 us on fp32 rows instead of 53, of 236 in all.
//
// A pair of CTAs computes 256 grouped rows (the MMA's M: 128 per CTA, one TMEM lane each) by 256 weight
// rows (N), each CTA loading its own rows and half of the weights (cta_group::2). A single CTA with 128 x 256
// tiles reads 51 KB from L2 for every 512 cycles of tensor work, more than an SM takes in; the pair needs 35 KB
// per CTA. For GATEUP the 256 are 128 gate rows (one CTA's half) and the same features' 128 up rows (the
// other's), so a thread of the epilogue holds a and b of one token for 128 features: it forms h, takes the
// largest magnitude of each 32 features in its own registers, and writes 16 bytes of codes and one scale byte per
// block, with no exchange between threads.
//
// Per 256 values of K (one ring stage per CTA: 16 KB of tokens, 16 KB of weights, 3 KB of scales): six
// tcgen05.cp bring the scales into TMEM, four columns per 128 rows and 128 values as the MMA wants them (the
// scale layout in memory is the one the copy reads; each CTA holds its own rows' scales and all 256 weight
// rows'), and four MMAs of K = 64 follow, each naming its pair of scale bytes in its instruction descriptor.
//
// TMEM has 512 columns and two 256-column accumulators would leave none for scales. The two accumulators
// overlap in 48 columns instead ([0, 256) and [208, 464), scales in [464, 512)): the epilogue reads the
// shared columns first and then lets the next tile's MMAs start.
//
// An expert with at most 128 rows left uses the first CTA's lanes only: the second CTA still brings its half
// of the weights, which at such sizes are the traffic. Rows past the routed ones are not loaded where a box of
// 32 rows can be spared; their lanes hold products of stale codes, which the epilogue replaces with zeros.
//
// Both kernels are launched as programmatic dependents (and the combine after DOWN is one, too): they may start while the
// kernel before them runs. What that one writes can be read only after the wait for it, and GATEUP may follow any
// kernel, so until then it sets up and asks for its first tile's weights in L2, by offsets that may yet change: a hint
// that stays within the weights whatever the offsets hold. After the wait it reads the offsets again, and lets DOWN start.
// DOWN thus finds offsets and weights final and brings its first tile's weights at once; it waits for GATEUP before it
// touches h or writes anything.
//
// Warp roles in both CTAs: warp 0 producer (TMA), warp 1 TMEM allocation and, in the leader, MMA issue,
// warps 2..9 epilogue (two warps per 32-lane TMEM quarter). The grid is persistent, at most one CTA per SM; every
// wait is bounded (0.2 s), on timeout the kernel records MOE_ERR_DEVICE_TIMEOUT in the workspace status word and
// leaves.
#include <atomic>

#include "fp4_gemm.cuh"

namespace moe {
namespace tc {
namespace fp4g {

constexpr int MT = 256;                       // grouped rows per tile, MC of them per CTA
constexpr int MC = 128;
constexpr int NT = 256;                       // weight rows per tile, half of them loaded by each CTA
constexpr int A_BYTES = MC * 128, B_BYTES = NT / 2 * 128;
constexpr int STAGE_BYTES = A_BYTES + B_BYTES + 3 * SF_BYTES;
// GATEUP writes codes straight from registers and gives all shared memory to the ring. DOWN stages its tile of y (64 KB
// per CTA) in 32 KB, one block of 32 x 64 per epilogue warp, and has five stages left; with 64 KB and four stages the
// whole FFN took 246 instead of 244 us at 8192 tokens, with plain 16-byte stores 250.
template <int K> struct Cfg {
  static constexpr int STAGES = K == GATEUP ? 6 : 5;
  static constexpr int BUF_BYTES = 4096;                     // 32 rows x 64 columns of y, 128-byte swizzle
  static constexpr int NBUF = K == GATEUP ? 0 : 1;           // per epilogue warp
  static constexpr int EPI_BYTES = EPI_WARPS * NBUF * BUF_BYTES;
  static constexpr int NBARS = 2 * STAGES + 3;
  static constexpr int SMEM = STAGES * STAGE_BYTES + EPI_BYTES + 1024 + 8 * NBARS + 16 + (int)sizeof(Plan);
  static_assert(SMEM <= 232448, "MXFP4 GEMM shared memory exceeds 227 KB");
};
static_assert(STAGE_BYTES % 1024 == 0, "ring stages keep the swizzle atoms' 1024-byte alignment");

constexpr uint32_t ACC1 = 208;                // first column of the second accumulator
constexpr uint32_t SF_COL = 464;              // scales: two sets of 8 (tokens) + 16 (weights) columns
constexpr uint32_t SF_SET = 24;

// Arrival (without release) on a barrier that may lie in the peer CTA. Announces that TMEM columns have been read:
// tcgen05.wait::ld has completed the reads and no memory is handed over. A releasing arrival would first
// wait for the warp's earlier global stores: 1300 to 3500 cycles in every tile here, with the tensor cores idle.
__device__ __forceinline__ void arrive_relaxed(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}
// tmA, tmA32: the token codes in boxes of 128 and of 32 rows; tmB: the weight codes, 128 rows; tmSA, tmSB: the
// scales, one stage of 128 rows per box; tmC: y (DOWN), blocks of 32 rows x 64 columns.
template <int K>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(THREADS, 1)
    fp4_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmA32,
               const __grid_constant__ CUtensorMap tmB, const __grid_constant__ CUtensorMap tmSA,
               const __grid_constant__ CUtensorMap tmSB, const __grid_constant__ CUtensorMap tmC, const Params p) {
  using C = Cfg<K>;
  constexpr int STAGES = C::STAGES;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t *epi_smem = smem + STAGES * STAGE_BYTES;
  uint64_t *bars = reinterpret_cast<uint64_t *>(epi_smem + C::EPI_BYTES);
  // bars: full[STAGES], empty[STAGES], tfull, tdrain (the shared columns have been read), mma_done
  uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(bars + C::NBARS);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_holder + 1);
  Plan &plan = *reinterpret_cast<Plan *>(tmem_holder + 4);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)cluster_ctarank();
  const bool leader = rank == 0;
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bar0 = smem_u32(bars);
  auto full_bar = [&](int s) { return bar0 + 8u * s; };              // the leader's counts both CTAs' bytes
  auto empty_bar = [&](int s) { return bar0 + 8u * (STAGES + s); };
  const uint32_t tfull_bar = bar0 + 8u * (2 * STAGES), tdrain_bar = tfull_bar + 8u, mma_done_bar = tfull_bar + 16u;

  if (K == DOWN) start_next();
  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    mbar_init(tfull_bar, 1);
    mbar_init(tdrain_bar, 2 * EPI_WARPS);
    mbar_init(mma_done_bar, 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    for (const CUtensorMap *m : {&tmB, &tmSB, &tmA, &tmA32, &tmSA})
      asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(m)) : "memory");
  }
  const int cluster_id = blockIdx.x >> 1, num_clusters = gridDim.x >> 1;
  if (warp == 0) {
    make_plan<MT>(p, lane, plan);
    if (K == GATEUP) {
      __syncwarp();
      Walker<MT> walk(cluster_id, num_clusters, p, plan);
      Tile t;
      if (walk.next(t, p, plan) && elect_one()) {
        const int w0 = t.e * p.w_rows_e + t.ft * p.w_step + (leader ? 0 : p.w_second);
        for (int kb = 0; kb < min(p.num_kb, STAGES); ++kb) {
          prefetch_2d(&tmB, kb * 128, w0);
          prefetch_2d(&tmSB, kb * (SF_BYTES / 4), w0 / 128);
        }
      }
      __syncwarp();
      wait_previous();
      make_plan<MT, true>(p, lane, plan);
    }
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_holder)),
                 "r"(512u)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  cluster_sync();   // both CTAs: barriers initialised, plan made, TMEM allocated
  if (K == GATEUP) start_next();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_holder;
  // routed rows of a tile among a CTA's 128, and the 32-row boxes that hold them (4: one box of 128)
  auto rows_of = [](const Tile &t, int r) { return min(MC, max(0, t.valid - MC * r)); };
  auto boxes_of = [](int rows) { return rows > MC / 2 ? 4 : (rows + 31) / 32; };

  if (warp == 0) {
    // ------------------------------------------------------------------ producer (both CTAs)
    int stage = 0, fills = 0;
    uint32_t phase = 0;
    bool ok = true;
    // one stage's weights and scales
    auto load_weights = [&](const Tile &t, int kb, int st) {
      const uint32_t sB = sbase + st * STAGE_BYTES + A_BYTES, sS = sB + B_BYTES, fb = mapa_shared(full_bar(st), 0);
      const int w0 = t.e * p.w_rows_e + t.ft * p.w_step, w1 = w0 + p.w_second;
      if (leader) {
        const int b0 = boxes_of(rows_of(t, 0)), b1 = boxes_of(rows_of(t, 1));
        mbar_expect_tx(full_bar(st), (uint32_t)(b0 + b1) * (A_BYTES / 4) + 2u * B_BYTES + (b1 ? 6u : 5u) * SF_BYTES);
      }
      tma_load_2d_pair(sB, &tmB, kb * 128, leader ? w0 : w1, fb);
      tma_load_2d_pair(sS + SF_BYTES, &tmSB, kb * (SF_BYTES / 4), w0 / 128, fb);
      tma_load_2d_pair(sS + 2 * SF_BYTES, &tmSB, kb * (SF_BYTES / 4), w1 / 128, fb);
    };
    auto load_tokens = [&](const Tile &t, int kb, int st) {
      const uint32_t sA = sbase + st * STAGE_BYTES, fb = mapa_shared(full_bar(st), 0);
      const int arow = t.start + MC * rank, boxes = boxes_of(rows_of(t, rank));
      if (boxes == 4) {
        tma_load_2d_pair(sA, &tmA, kb * 128, arow, fb);
      } else {
        for (int b = 0; b < boxes; ++b) tma_load_2d_pair(sA + b * (A_BYTES / 4), &tmA32, kb * 128, arow + 32 * b, fb);
      }
      if (boxes) tma_load_2d_pair(sA + A_BYTES + B_BYTES, &tmSA, kb * (SF_BYTES / 4), arow / 128, fb);
    };
    Walker<MT> walk(cluster_id, num_clusters, p, plan);
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
        if (!mbar_spin_cluster(empty_bar(stage), phase ^ 1u, abort_flag, p.hdr, 41)) { ok = false; break; }
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
    if (leader && *abort_flag) {
      // leave no copy in flight: wait (bounded) for the last fill of every stage; the peer, whose bytes arrive on
      // the same barriers, stays until the cluster meets below
      const uint64_t t0 = global_ns();
      for (int i = 1; i <= STAGES && i <= fills; ++i) {
        const int f = fills - i;   // fill number f went to stage f % STAGES in ring round f / STAGES
        while (!mbar_try_wait(full_bar(f % STAGES), (uint32_t)(f / STAGES) & 1u) && global_ns() - t0 < kWaitLimitNs) {}
      }
    }
  } else if (warp == 1 && leader) {
    // ------------------------------------------------------------------ MMA issuer (leader only)
    wait_previous();
    int stage = 0, n = 0, set = 0;
    uint32_t phase = 0;
    bool issued = false, ok = true;
    const uint64_t desc_a0 = sdesc(sbase, 16, 1024), desc_b0 = sdesc(sbase + A_BYTES, 16, 1024);
    const uint64_t desc_s0 = sf_desc(sbase + A_BYTES + B_BYTES);
    Walker<MT> walk(cluster_id, num_clusters, p, plan);
    for (Tile t; ok && walk.next(t, p, plan); ++n) {
      if (n > 0 && !mbar_spin_cluster(tdrain_bar, (uint32_t)(n - 1) & 1u, abort_flag, p.hdr, 42)) break;
      tc_fence_after();
      const uint32_t d = tmem_base + ((n & 1) ? ACC1 : 0u);
      for (int kb = 0; kb < p.num_kb; ++kb) {
        if (!mbar_spin_cluster(full_bar(stage), phase, abort_flag, p.hdr, 43)) { ok = false; break; }
        tc_fence_after();
        if (elect_one()) {
          const uint32_t so = (uint32_t)(stage * STAGE_BYTES) >> 4;
          const uint32_t sfa = tmem_base + SF_COL + (uint32_t)set * SF_SET, sfb = sfa + 8;
#pragma unroll
          for (int h = 0; h < 2; ++h) {   // 128 values of K each
            copy_scales<2>(sfa + 4 * h, desc_s0 + so + (uint32_t)((h * 512) >> 4));
            copy_scales<2>(sfb + 8 * h, desc_s0 + so + (uint32_t)((SF_BYTES + h * 512) >> 4));
            copy_scales<2>(sfb + 8 * h + 4, desc_s0 + so + (uint32_t)((2 * SF_BYTES + h * 512) >> 4));
#pragma unroll
            for (int kk = 0; kk < 2; ++kk) {
              const uint32_t koff = (uint32_t)((2 * h + kk) * 32) >> 4;
              mma_mxf4<2>(d, desc_a0 + so + koff, desc_b0 + so + koff, idesc(MT, NT, 2u * kk), sfa + 4 * h, sfb + 8 * h,
                       (kb | h | kk) != 0 ? 1u : 0u);
            }
          }
          mma_commit_pair(empty_bar(stage), 0x3);   // frees the stage in both CTAs
        }
        __syncwarp();
        issued = true;
        set ^= 1;
        if (++stage == STAGES) { stage = 0; phase ^= 1u; }
      }
      if (!ok) break;
      if (elect_one()) mma_commit_pair(tfull_bar, 0x3);
      __syncwarp();
    }
    if (issued) {   // every MMA is done before TMEM is freed
      if (elect_one()) mma_commit_pair(mma_done_bar, 0x1);
      __syncwarp();
      const uint64_t t0 = global_ns();
      while (!mbar_try_wait(mma_done_bar, 0) && global_ns() - t0 < kWaitLimitNs) {}
    }
  } else if (warp >= 2) {
    // ------------------------------------------------------------------ epilogue
    wait_previous();
    const int quarter = warp & 3, hh = (warp - 2) >> 2;
    const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
    const uint32_t buf = smem_u32(epi_smem) + (uint32_t)(warp - 2) * (C::NBUF * C::BUF_BYTES);
    int n = 0;
    Walker<MT> walk(cluster_id, num_clusters, p, plan);
    for (Tile t; walk.next(t, p, plan); ++n) {
      if (!mbar_spin_cluster(tfull_bar, (uint32_t)n & 1u, abort_flag, p.hdr, 44)) break;
      tc_fence_after();
      const bool second = n & 1;
      const uint32_t tacc = tmem_base + lane_off + (second ? ACC1 : 0u);
      const int r_in = quarter * 32 + lane;                 // row among this CTA's 128
      const int valid = rows_of(t, rank), row0 = t.start + MC * rank;
      if (valid == 0) {   // the second CTA of a tile of at most 128 rows: nothing to write, not even padding
        if (lane == 0) arrive_relaxed(mapa_shared(tdrain_bar, 0));
        continue;
      }
      const bool real = r_in < valid;
      // the columns shared with the other accumulator come first: the last 48 of the first
      // accumulator, the first 48 of the second
      if (K == GATEUP) {
        const int64_t row = (int64_t)row0 + r_in;
#pragma unroll 1
        for (int i = 0; i < 2; ++i) {
          const int b = second ? 2 * i + hh : 3 - 2 * i - hh;   // block of 32 features
          uint32_t ra[32], rb[32];
          // shared: up rows of the first accumulator, gate rows of the second. Read alone, and handed over before the
          // other half is read: 237.9 against 240.0 us for the FFN at 8192 tokens.
          if (i == 0) {
            if (second) tmem_ld32(tacc + 32u * b, ra);
            else tmem_ld32(tacc + 128u + 32u * b, rb);
            tmem_ld_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive_relaxed(mapa_shared(tdrain_bar, 0));
            if (second) tmem_ld32(tacc + 128u + 32u * b, rb);
            else tmem_ld32(tacc + 32u * b, ra);
          } else {
            tmem_ld32(tacc + 32u * b, ra);
            tmem_ld32(tacc + 128u + 32u * b, rb);
          }
          tmem_ld_wait();
          // sigmoidf_ (__expf: 2 + 1.17 |z| ulp, and an approximate reciprocal) is off by a few 2^-23 here, where a comes from
          // fp32 sums and h goes to 4 bits: of the order of the sums' own error, so that a value within it of a
          // rounding threshold may get the neighbouring code.
          float hv[32], top = 0.0f;
#pragma unroll
          for (int c = 0; c < 32; c += 2) {
            const float a0 = __uint_as_float(ra[c]), a1 = __uint_as_float(ra[c + 1]);
            hv[c] = a0 * __uint_as_float(rb[c]) * sigmoidf_(a0);
            hv[c + 1] = a1 * __uint_as_float(rb[c + 1]) * sigmoidf_(a1);
            // largest magnitude; a NaN stays
            asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(top) : "f"(hv[c]), "f"(hv[c + 1]), "f"(top));
          }
          uint32_t byte = fp4::scale_byte(__float_as_uint(top) & 0x7fffffffu);
          const float inv = fp4::inv_scale(byte);
          uint32_t q[4];
#pragma unroll
          for (int c = 0; c < 32; ++c) hv[c] *= inv;
#pragma unroll
          for (int c = 0; c < 4; ++c) q[c] = fp4::pack_e2m1x8(hv + 8 * c);
          if (!real || byte == 255u) q[0] = q[1] = q[2] = q[3] = 0u;
          if (!real) byte = 0u;
          if (row < p.rows_max) {
            *reinterpret_cast<uint4 *>(p.h + row * (p.f / 2) + t.ft * 64 + 16 * b) = make_uint4(q[0], q[1], q[2], q[3]);
            p.h_scales[fp4::scale_word(row, t.ft, p.f / 128) + b] = (uint8_t)byte;
          }
        }
      } else {
#pragma unroll 1
        for (int i = 0; i < 2; ++i) {
          const int c4 = second ? 2 * i + hh : 3 - 2 * i - hh;   // block of 64 columns
          uint32_t r[64];
          tmem_ld32(tacc + 64u * c4, *reinterpret_cast<uint32_t(*)[32]>(r));
          tmem_ld32(tacc + 64u * c4 + 32u, *reinterpret_cast<uint32_t(*)[32]>(r + 32));
          tmem_ld_wait();
          if (i == 0) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive_relaxed(mapa_shared(tdrain_bar, 0));
          }
          if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");   // the last store has read the block
          __syncwarp();
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            uint32_t w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
              w[j] = real ? pack_bf16x2(__uint_as_float(r[8 * q + 2 * j]), __uint_as_float(r[8 * q + 2 * j + 1])) : 0u;
            const uint32_t addr = buf + (uint32_t)lane * 128 + ((uint32_t)(q ^ (lane & 7)) << 4);
            asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3])
                         : "memory");
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          if (lane == 0) {
            asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                             reinterpret_cast<uint64_t>(&tmC)),
                         "r"(t.ft * NT + 64 * c4), "r"(row0 + quarter * 32), "r"(buf)
                         : "memory");
            asm volatile("cp.async.bulk.commit_group;" ::: "memory");
          }
        }
      }
    }
    if (K == DOWN && lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    __syncwarp();
  }

  tc_fence_before();
  cluster_sync();   // no CTA leaves while its peer may still signal its barriers or use its TMEM
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(512u) : "memory");
  }
}

// The kernel's dynamic shared memory limit, raised once per device (the call costs a host microsecond).
template <int K> static bool smem_allowed() {
  static std::atomic<uint64_t> done{0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return false;
  if (dev < 64 && (done.load(std::memory_order_relaxed) >> dev & 1)) return true;
  if (cudaFuncSetAttribute(fp4_kernel<K>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<K>::SMEM) != cudaSuccess) {
    (void)cudaGetLastError();
    return false;
  }
  if (dev < 64) done.fetch_or((uint64_t)1 << dev, std::memory_order_relaxed);
  return true;
}

constexpr int kFewRows = 48;

template <int K>
static int launch(const Maps &m, const Params &p, cudaStream_t s) {
  if (!smem_allowed<K>()) return MOE_ERR_CUDA;
  int64_t clusters = sm_count() / 2;
  const int64_t most = p.rows_max / MC * p.n_ft;   // tiles there can be
  if (most < clusters) clusters = most;
  MOE_TRY_CUDA(launch_after(fp4_kernel<K>, dim3((unsigned)(2 * clusters)), dim3(THREADS), Cfg<K>::SMEM, s, m.a, m.a32,
                            m.b, m.sa, m.sb, m.c, p));
  return MOE_OK;
}

}  // namespace fp4g
}  // namespace tc
}  // namespace moe

using namespace moe;

extern "C" int moe_grouped_ffn_fwd_fp4(const void *x_codes, const void *x_scales, const void *wgu_codes,
                                       const void *wgu_scales, const void *wd_codes, const void *wd_scales,
                                       const int32_t *tile_offsets, const int32_t *offsets, int E, int d, int f,
                                       int64_t rows_max, void *h_codes, void *h_scales, void *y_perm, void *ws,
                                       size_t ws_bytes, moe_stream_t stream) {
  using namespace tc::fp4g;
  if (E < 1 || E > MOE_MAX_EXPERTS || d < 1 || f < 1 || rows_max < 0 || rows_max % MOE_GROUP_ROWS)
    return MOE_ERR_INVALID_ARG;
  if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255) ||
      ws_bytes < moe_grouped_ffn_workspace_size(E, d, f, rows_max, MOE_BF16, 0))
    return MOE_ERR_INVALID_ARG;
  if (d % 256 || f % 256 || rows_max >= ((int64_t)1 << 31) || (int64_t)E * 2 * f >= ((int64_t)1 << 31) ||
      (int64_t)E * d >= ((int64_t)1 << 31))
    return MOE_ERR_UNSUPPORTED;
  if (rows_max == 0) return MOE_OK;
  const void *ptrs[] = {x_codes, x_scales, wgu_codes, wgu_scales, wd_codes, wd_scales, h_codes, h_scales, y_perm};
  for (const void *q : ptrs)
    if (!q || !aligned16(q)) return MOE_ERR_INVALID_ARG;
  if (!tile_offsets || !offsets) return MOE_ERR_INVALID_ARG;
  cudaStream_t s = (cudaStream_t)stream;
  Maps m{};
  Params p{};
  p.tile_offsets = tile_offsets;
  p.offsets = offsets;
  p.hdr = static_cast<WsHeader *>(ws);
  p.E = E;
  p.rows_max = rows_max;
  p.d = d;
  p.f = f;
  p.y = (__nv_bfloat16 *)y_perm;
  // Which kernels: by the routed rows per expert, at most rows_max / E less the padding. From tokens to combined output
  // at d = 2048, E = 64, k = 8, f = 1024, those for few rows against these: 0.1 rows per expert 20.7 and 24.8 us, 1 row
  // 41.0 and 46.1, 8 rows 55.3 and 60.2, 42 rows 62.0 and 64.8, 64 rows 66.9 and 64.9, 128 rows 83.7 and 70.5.
  const bool few = rows_max / E - (MOE_GROUP_ROWS - 1) <= kFewRows;

  // (the kernels for few rows read tokens in boxes of 32 rows only and store y without a map)
  if (!(few || codes_map(&m.a, x_codes, rows_max, d / 2, MC)) || !codes_map(&m.a32, x_codes, rows_max, d / 2, 32) ||
      !codes_map(&m.b, wgu_codes, (uint64_t)E * 2 * f, d / 2, 128) || !scales_map(&m.sa, x_scales, rows_max, d) ||
      !scales_map(&m.sb, wgu_scales, (uint64_t)E * 2 * f, d))
    return MOE_ERR_CUDA;
  m.c = m.b;   // not used
  p.n_ft = f / 128;
  p.num_kb = d / KS;
  p.w_rows_e = 2 * f;
  p.w_second = f;
  p.w_step = 128;
  p.h = (uint8_t *)h_codes;
  p.h_scales = (uint8_t *)h_scales;
  int rc = few ? few_gateup(m, p, s) : launch<GATEUP>(m, p, s);
  if (rc) return rc;

  if (!(few || codes_map(&m.a, h_codes, rows_max, f / 2, MC)) || !codes_map(&m.a32, h_codes, rows_max, f / 2, 32) ||
      !codes_map(&m.b, wd_codes, (uint64_t)E * d, f / 2, 128) || !scales_map(&m.sa, h_scales, rows_max, f) ||
      !scales_map(&m.sb, wd_scales, (uint64_t)E * d, f) || !(few || tc::make_map(&m.c, y_perm, rows_max, d, 32)))
    return MOE_ERR_CUDA;
  p.n_ft = d / NT;
  p.num_kb = f / KS;
  p.w_rows_e = d;
  p.w_second = 128;
  p.w_step = NT;
  return few ? few_down(m, p, s) : launch<DOWN>(m, p, s);
}
