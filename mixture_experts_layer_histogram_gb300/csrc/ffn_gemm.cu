// The gated feed-forward block's matrix products in bf16 on CTA pairs (sm_103a, tcgen05.mma.cta_group::2).
//
//   GATEUP  [a | b] = x [Wg | Wu]^T; the epilogue forms h = act(a) b from the fp32 accumulators, and keeps a, b (bf16, or
//           8-bit codes with a power of two per 32 values) where a backward follows
//   DOWN    y = h Wd^T (+ y_in)
//   DH      dh = dy Wd; the epilogue reads the kept a, b and writes da = dh b act'(a), db = dh act(a) (from 8-bit codes also
//           h again, which the weight gradient needs)
//   BACK    dx = [da | db] [Wg; Wu] (+ dx_in), dWgu = [da | db]^T x and dWd = dy^T h (both operands read MN-major)
//
// A pair computes 256 x 256 outputs: each CTA holds 128 rows of A and half of B's 256 rows per 64-deep ring stage (32 KB for
// 256 x 256 x 64 x 2 flops a pair, the ratio of bytes to flops at which the L2 just keeps up) and 128 x 256 accumulators
// in its own TMEM, twice (512 columns), so the epilogue of one tile runs beside the products of the next.
// GATEUP's B is 128 gate rows in one CTA and the same features' 128 up rows in the other: every thread of the epilogue
// (a TMEM lane is a token) holds a and b of the same features, a whole block of 32 at a time for the 8-bit codes.
//
// One launch runs all products of a call: y's tiles follow the ones of h in the same kernel, the last three products those of
// da, db. A pair takes its tiles in the order of the products, as many of each as even out the pairs' work (deal_out); a unit
// that reads what others of the launch write waits until the rows of tiles that it needs are complete (counts per row, in the
// workspace; the pairs are all resident, a cooperative launch, and no pair waits before it has brought all its tiles of the
// first product). In separate launches the incomplete last rounds, the set-up of each kernel and its last epilogues cost 45 of
// 259 us of a step at 8192 x 2048 x 1024.
//
// A product of fewer tiles than pairs gets more of them: tiles of 128 columns instead of 256, or its tiles cut along K into S
// parts (plan). The warps that hold the parts of the same outputs leave their fp32 accumulators in the workspace, wait until all
// are there (every pair is resident, and takes its parts in the order of their tiles, so that ends) and finish a share of the
// outputs each, adding the parts up in their order. (One warp finishing all of them took 22 us for eight parts.) 389 x 2048 x
// 1024 forward: 26.6 us in two launches of wide tiles, 22.5 in one with narrow ones. Of the 18.5 us inside the kernel, 2.7 pass
// before the first product starts, 3 and 2.8 in the products, 3.8 in the exchange of parts, 2.4 between the last row of h and
// the sight of it. There, proxy fences for all memory instead of global memory alone had cost 2 us more.
//
// Roles per CTA: warp 0 loads (TMA), warp 1 allocates TMEM and, in the leader, issues the products, warps 2..9 are the epilogue
// (sixteen warps of 96 registers were slower: 1474 against 1400 us for the three products at 8192 x 4096 x 8192).
// Every wait is bounded (0.2 s): on timeout the kernel records MOE_ERR_DEVICE_TIMEOUT, lets copies in flight land, frees
// TMEM and leaves.
//
// Measured (bf16, T x d x f): 8192 x 4096 x 8192 with 8 bits kept, forward 0.87 ms, backward 1.73-1.78 ms each alone at full
// clocks (1.91 PFLOP/s; the tensor pipe is busy 89% of the time), a step under the power cap 2.95-3.05 ms (1.65 PFLOP/s, of 1.75
// that a long library product holds); 8192 x 2048 x 1024 forward 67 us, backward 126-130 us (tensor pipe 67% and 74%), a step
// 196 us in short runs and 214 under the cap: per tile the products take 8.6 us, but bursts of h, a, b and da, db from all pairs
// at once take 4-7 us of HBM's time each, and each launch 2.7 us to its first product and 3 us from its last.
#include <cuda.h>

#include <string.h>

#include <algorithm>
#include <atomic>
#include <type_traits>
#include <utility>

#include "f32x2.cuh"
#include "ffn.cuh"
#include "tc_ptx.cuh"
#include "tma_host.cuh"

namespace moe {
namespace tc {
namespace ffng {

using ffn::Gate;

enum Chain { FWD = 0, BWD = 1 };                     // the kernel's two instantiations, and
enum Op { GATEUP = 0, DOWN = 1, DH = 2, DW = 3, DX = 4 };   // the products they run

constexpr int TILE = 256;                       // rows and columns of a pair's tile
constexpr int HALF = TILE / 2;                  // a CTA's rows of A, and of B
constexpr int BK = 64;
constexpr int OPERAND = HALF * BK * 2;          // bytes of one operand per stage
constexpr int STAGE = 2 * OPERAND;
constexpr int STAGES = 5;
constexpr int EPI_WARPS = 8;
constexpr int THREADS = 64 + 32 * EPI_WARPS;
constexpr int BUF = 32 * 64 * 2;                // a block of 32 rows x 64 columns; every epilogue warp has two
constexpr int NBARS = 2 * STAGES + 5;
constexpr int SMEM = STAGES * STAGE + EPI_WARPS * 2 * BUF + 1024 + 8 * NBARS + 16;
static_assert(SMEM <= 232448, "shared memory exceeds 227 KB");
constexpr int SLICES = 2 * EPI_WARPS;           // of a tile: one per epilogue warp of the pair, 32 rows x 128 columns
constexpr int SLICE_FLOATS = 32 * HALF;
constexpr int MAX_SPLIT = 8;

// One matrix product
enum Needs { NOTHING = 0, ITS_ROWS = 1, ALL_ROWS = 2 };   // of what an earlier product of the same launch writes
struct Product {
  int op, needs;
  int M, N;                  // valid rows; valid columns (GATEUP, DH: f)
  int width;                 // columns of a tile: 256 or 128
  int m_tiles, n_tiles, num_kb;
  int splits;                // its tiles are cut along K into this many parts (1: whole tiles)
  int first, at;             // splits > 1: the pair that has the first part; the tiles' place in `part` and `arrived`
  __nv_bfloat16 *out0;       // GATEUP: kept ab (null: not kept, or in 8 bits); DH: dab; else the result
  __nv_bfloat16 *out1;       // GATEUP: h; DH from 8 bits: h
  const __nv_bfloat16 *in0;  // DH: kept ab; DOWN, DX: what is added (null: nothing)
};
constexpr int PRODUCTS = 4;
template <int CH> constexpr int products() { return CH == FWD ? 2 : PRODUCTS; }
template <int CH> struct Maps {
  CUtensorMap a[products<CH>()], b[products<CH>()];
};
constexpr int MAX_PAIRS = 96;   // a warp holds the pairs' counts, three a lane
struct Params {
  WsHeader *hdr;
  // The products in the order in which every pair takes its tiles of them, and how many of each it gets; deal: the order in which
  // the host deals them out
  int products, deal[PRODUCTS];
  Product prod[PRODUCTS];
  uint16_t count[PRODUCTS][MAX_PAIRS];
  // Tiles that are cut along K
  float4 *part;              // [place + part][slice][32][32] float4
  int *arrived;              // [place][slice][2]: parts written, warps done with them
  // Rows of tiles that the launch's first product has written: warps arrived per row, and what makes a row complete
  int *ready, *left;         // left: pairs that are done (the last one sets ready back to zero)
  int rows, row_need;
  Gate gate;
  uint8_t *codes, *scales;   // GATEUP, DH: ab in 8 bits (null: bf16)
};

// One unit of work: a tile and its k-blocks.
struct Unit {
  int q;                     // product
  int tile, m, n, kb0, kb1;
  int part;                  // -1: the whole tile
};

// Tiles are numbered in bands of eight rows of tiles, column by column inside a band: the tiles that run at the same
// time share few rows of A and few columns of B.
constexpr int BAND = 8;
__device__ __forceinline__ void place(Unit &t, const Product &o) {
  const int per = BAND * o.n_tiles, band = t.tile / per, r = t.tile - band * per;
  const int height = min(BAND, o.m_tiles - band * BAND);
  t.n = r / height;
  t.m = band * BAND + (r - t.n * height);
}

// The units of one pair, in order; the whole warp walks. In round t of a product the pairs that have more than t of its tiles
// take consecutive ones; parts of cut tiles go round all pairs.
struct Walk {
  int pair, pairs, c, t, base;   // cut: t is the next part's number
  int n0, n1, n2;            // this lane's share of the product's counts
  __device__ __forceinline__ Walk(int pair_, int pairs_, const Params &p) : pair(pair_), pairs(pairs_), c(0) { open(p); }
  // (Loads of the parameters through their generic address: one per 32 lanes, where the constant path takes them lane by lane.)
  static __device__ __forceinline__ int count(const uint16_t *at) {
    uint16_t v;
    asm volatile("ld.u16 %0, [%1];" : "=h"(v) : "l"(at));
    return v;
  }
  __device__ __forceinline__ void open(const Params &p) {
    const uint16_t *row = p.count[c] + (threadIdx.x & 31);
    t = base = 0;
    if (p.prod[c].splits > 1) {
      t = pair - p.prod[c].first;
      if (t < 0) t += pairs;
    }
    n0 = count(row);
    n1 = count(row + 32);
    n2 = count(row + 64);
  }
  __device__ __forceinline__ bool next(Unit &w, const Params &p) {
    w.part = -1;
    for (;;) {
      const Product &o = p.prod[c];
      if (o.splits > 1) {
        if (t < o.m_tiles * o.n_tiles * o.splits) {
          w.tile = t / o.splits;
          w.part = t - w.tile * o.splits;
          t += pairs;
          break;
        }
      } else {
        const uint32_t b0 = __ballot_sync(0xffffffffu, n0 > t), b1 = __ballot_sync(0xffffffffu, n1 > t),
                       b2 = __ballot_sync(0xffffffffu, n2 > t);
        const uint32_t mine = pair < 32 ? b0 : (pair < 64 ? b1 : b2), below = (1u << (pair & 31)) - 1;
        if (mine >> (pair & 31) & 1) {
          w.tile = base + __popc(mine & below) + (pair >= 32 ? __popc(b0) : 0) + (pair >= 64 ? __popc(b1) : 0);
          base += __popc(b0) + __popc(b1) + __popc(b2);
          ++t;
          break;
        }
      }
      if (++c >= p.products) return false;
      open(p);
    }
    const Product &o = p.prod[w.q = c];
    w.kb0 = w.part < 0 ? 0 : (int)((int64_t)o.num_kb * w.part / o.splits);
    w.kb1 = w.part < 0 ? o.num_kb : (int)((int64_t)o.num_kb * (w.part + 1) / o.splits);
    place(w, o);
    return true;
  }
};

// kind::f16: D fp32, A and B bf16, M = 256, N = width
__device__ __forceinline__ uint32_t idesc(bool a_mn, bool b_mn, int width) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) |
         ((uint32_t)(width >> 3) << 17) | ((uint32_t)(TILE >> 4) << 24);
}

// TMEM has been read (wait::ld): nothing in memory is handed over, so the arrival need not wait for this warp's stores
__device__ __forceinline__ void arrive_leader(uint32_t bar) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(mapa_shared(bar, 0)) : "memory");
}

// The waits below are made by whole warps. Lanes look for themselves, but go on, or give up, together: one that went on alone would
// wait for the others at the warp's next barrier for good.
__device__ __forceinline__ bool given_up(uint64_t t0, volatile int *abort_flag, WsHeader *hdr, int where) {
  const bool late = global_ns() - t0 > kWaitLimitNs;
  if (!__any_sync(0xffffffffu, late || *abort_flag)) return false;
  if (late) report(hdr, MOE_ERR_DEVICE_TIMEOUT, where);
  *abort_flag = 1;
  return true;
}
// Polling, for the ring's producer and the MMA issuer (see mbar_spin_cluster) ...
__device__ __forceinline__ bool spin_warp(uint32_t bar, uint32_t parity, volatile int *abort_flag, WsHeader *hdr, int where) {
  const uint64_t t0 = global_ns();
  for (uint32_t i = 0;; ++i) {
    if (__all_sync(0xffffffffu, mbar_ready_cluster(bar, parity))) return true;
    if ((i & 255u) == 255u && given_up(t0, abort_flag, hdr, where)) return false;
  }
}
// ... and for the others, in place: across a call, what a warp has asked for ahead would be stored to the stack first, and so waited
// for.
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, volatile int *abort_flag, WsHeader *hdr, int where) {
  const uint64_t t0 = global_ns();
  for (uint32_t i = 0;; ++i) {
    if (__all_sync(0xffffffffu, mbar_try_wait_cluster(bar, parity))) return true;
    if ((i & 15u) == 15u && given_up(t0, abort_flag, hdr, where)) return false;
  }
}

// Bounded wait of a whole warp until *count is n; what was written before the counts is then visible.
__device__ __forceinline__ bool wait_count(const int *count, int n, volatile int *abort_flag, WsHeader *hdr) {
  const uint64_t t0 = global_ns();
  for (;;) {
    int v;
    asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(count) : "memory");
    if (__all_sync(0xffffffffu, v == n)) return true;
    const bool late = global_ns() - t0 > kWaitLimitNs;
    if (__any_sync(0xffffffffu, late || *abort_flag)) {
      if (late) report(hdr, MOE_ERR_DEVICE_TIMEOUT, 45);
      *abort_flag = 1;
      return false;
    }
  }
}

// What the producer knows of the rows that its units read.
struct Rows {
  bool all = false;          // every row is written
  // One look. What it finds written is ordered before the TMA's reads.
  __device__ __forceinline__ bool look(const Params &p, const Product &o, int m) {
    if (o.needs == NOTHING || all) return true;
    bool there = true;
    const int lane = threadIdx.x & 31;
    if (o.needs == ITS_ROWS) {
      there = arrived(p.ready + m) == p.row_need;
    } else {
      for (int r = lane; r < p.rows; r += 32) there = there && arrived(p.ready + r) == p.row_need;
    }
    there = __all_sync(0xffffffffu, there);
    if (there) {
      asm volatile("fence.proxy.async.global;" ::: "memory");
      all = o.needs == ALL_ROWS;
    }
    return there;
  }
  static __device__ __forceinline__ int arrived(const int *at) {
    int v;
    asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(at) : "memory");
    return v;
  }
  __device__ __forceinline__ bool wait(const Params &p, const Product &o, int m, volatile int *abort_flag) {   // bounded
    const uint64_t t0 = global_ns();
    while (!look(p, o, m)) {
      const bool late = global_ns() - t0 > kWaitLimitNs;
      if (__any_sync(0xffffffffu, late || *abort_flag)) {
        if (late) report(p.hdr, MOE_ERR_DEVICE_TIMEOUT, 46);
        *abort_flag = 1;
        return false;
      }
    }
    return true;
  }
};

// Blocks on their way out and in. A warp holds 32 rows, one per lane; global memory wants consecutive bytes of a row from
// neighbouring lanes. Blocks therefore pass through shared memory, W = 64 columns wide (128 bytes a row, eight lanes) or 32 (64
// bytes, four lanes), 16-byte chunks XOR-swizzled so that neither side meets bank conflicts. (Straight from a row per lane, 32
// bytes each, needs no shared memory, but 32 lines per instruction slow the ring's own copies: in launches of their own 38
// against 33 us for y at 8192 x 2048 x 1024, 52 against 43 for da, db.) Rows from `rows` and columns from `cols` on are left
// out, and read as zero.
template <int W> struct Chunk {
  static constexpr int LANES = W / 8, STEP = 32 / LANES, N = W / 8;   // lanes per row, rows per instruction, instructions
  static __device__ __forceinline__ uint32_t at(uint32_t buf, int row, int chunk) {
    const uint32_t sw = W == 64 ? (uint32_t)row & 7u : ((uint32_t)row >> 1) & 3u;
    return buf + (uint32_t)row * (2 * W) + (((uint32_t)chunk ^ sw) << 4);
  }
};
__device__ __forceinline__ void st_shared_v4(uint32_t a, const uint4 &q) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(q.x), "r"(q.y), "r"(q.z), "r"(q.w) : "memory");
}
// N chunks of 8 columns of this lane's row (from chunk c0 on) into the buffer
template <int W, int N> __device__ __forceinline__ void stage(uint32_t buf, int lane, int c0, const float *v) {
#pragma unroll
  for (int c = 0; c < N; ++c) st_shared_v4(Chunk<W>::at(buf, lane, c0 + c), pack_bf16x8(v + 8 * c));
}
// The buffer's block to rows row0.. and columns col.. of a row-major output
template <int W>
__device__ __forceinline__ void put(uint32_t buf, int lane, __nv_bfloat16 *out, int64_t ld, int row0, int rows, int col, int cols) {
  using C = Chunk<W>;
  __syncwarp();
  const int c = lane % C::LANES, r0 = lane / C::LANES;
  __nv_bfloat16 *dst = out + (int64_t)(row0 + r0) * ld + col + 8 * c;
#pragma unroll
  for (int i = 0; i < C::N; ++i) {
    const int r = r0 + C::STEP * i;
    const uint4 q = ld_shared_v4(C::at(buf, r, c));
    if (row0 + r < rows && col + 8 * c < cols) *reinterpret_cast<uint4 *>(dst + (int64_t)(C::STEP * i) * ld) = q;
  }
  __syncwarp();
}
// A block of an input into the buffer, copied by neighbouring lanes (asynchronously; zeros for what lies outside)
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void landed() {   // all but the last N groups of every lane
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
  __syncwarp();
}
template <int W>
__device__ __forceinline__ void fetch(uint32_t buf, const __nv_bfloat16 *in, int64_t ld, int row0, int rows, int col, int cols, int lane) {
  using C = Chunk<W>;
  const int c = lane % C::LANES, r0 = lane / C::LANES;
  const __nv_bfloat16 *src = in + (int64_t)(row0 + r0) * ld + col + 8 * c;
#pragma unroll
  for (int i = 0; i < C::N; ++i) {
    const int r = r0 + C::STEP * i;
    const bool there = row0 + r < rows && col + 8 * c < cols;
    copy16(C::at(buf, r, c), there ? src + (int64_t)(C::STEP * i) * ld : in, there);
  }
}
// This lane's row of the buffer: N chunks of 8 columns from chunk c0 on
template <int W, int N, bool ADD> __device__ __forceinline__ void take(uint32_t buf, int lane, int c0, float *v) {
#pragma unroll
  for (int c = 0; c < N; ++c) {
    float w[8];
    unpack_bf16x8(ld_shared_v4(Chunk<W>::at(buf, lane, c0 + c)), w);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[8 * c + i] = ADD ? v[8 * c + i] + w[i] : w[i];
  }
}
// The same for a 32 x 32 block of codes: two lanes per row.
__device__ __forceinline__ uint32_t code_at(uint32_t buf, uint32_t row, uint32_t half) { return buf + row * 32 + ((half ^ ((row >> 2) & 1u)) << 4); }
__device__ __forceinline__ void fetch_codes(uint32_t buf, const uint8_t *in, int64_t ld, int row0, int rows, int col, int cols, int lane) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = (lane >> 1) + 16 * i;
    const bool there = row0 + r < rows && col < cols;
    copy16(code_at(buf, r, lane & 1), there ? in + (int64_t)(row0 + r) * ld + col + 16 * (lane & 1) : in, there);
  }
}
__device__ __forceinline__ void unpack_codes(const uint4 &w, float scale, float *v) {   // 16 of them
  act8::unpack4(w.x, v);
  act8::unpack4(w.y, v + 4);
  act8::unpack4(w.z, v + 8);
  act8::unpack4(w.w, v + 12);
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] *= scale;
}

// 32 values, one whole block, to their codes and scale
__device__ __forceinline__ void put_block8(uint8_t *codes, uint8_t *scale, const float *v) {
  float top = 0.0f;
#pragma unroll
  for (int i = 0; i < 32; i += 2) top = act8::larger(top, v[i], v[i + 1]);
  const uint32_t byte = act8::scale_byte(__float_as_uint(top));
  const float inv = act8::inv_scale(byte);
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    w[i] = act8::pack4(v[4 * i] * inv, v[4 * i + 1] * inv, v[4 * i + 2] * inv, v[4 * i + 3] * inv);
    if (byte == 255u) w[i] = 0;
  }
  reinterpret_cast<uint4 *>(codes)[0] = make_uint4(w[0], w[1], w[2], w[3]);
  reinterpret_cast<uint4 *>(codes)[1] = make_uint4(w[4], w[5], w[6], w[7]);
  *scale = (uint8_t)byte;
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

// The warp's 32 x width / 2 accumulated outputs of a tile (GATEUP: a of width / 4 features, and b of the same)
template <int K> struct Slice {
  uint32_t tmem;             // TMEM address of the first column
  int apart;                 // GATEUP: columns from a to b
  __device__ __forceinline__ void load(int c, float *v) const {   // 16 columns from column c on
    uint32_t r[16];
    tmem_ld16(tmem + (uint32_t)c, r);
    tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
  }
};

// What an epilogue warp reads besides the accumulators is on its way to shared memory while the products still run: what is added
// (both its blocks), or the kept a and b of its first two blocks (the others follow as the buffers get free); scales in
// registers. (Loads into registers instead: what did not fit there was waited for before it could be put on the stack.)
template <int K> struct Ahead {
  uint32_t sa, sb;           // DH from 8 bits: the blocks' scales, a byte each
  static __device__ __forceinline__ void block(const Params &p, const Product &o, uint32_t buf, int lane, int row0, int col) {   // DH: a, b
    const int64_t ld = 2 * (int64_t)o.N;
    if (p.codes) {
      fetch_codes(buf, p.codes, ld, row0, o.M, col, o.N, lane);
      fetch_codes(buf + 1024, p.codes + o.N, ld, row0, o.M, col, o.N, lane);
    } else {
      fetch<32>(buf, o.in0, ld, row0, o.M, col, o.N, lane);
      fetch<32>(buf + 2048, o.in0 + o.N, ld, row0, o.M, col, o.N, lane);
    }
    commit();
  }
  __device__ __forceinline__ void start(const Params &p, const Product &o, uint32_t buf, int lane, int row0, int col0) {
    if (K == DOWN || K == DX) {
      if (o.in0) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          if (128 * j < o.width) fetch<64>(buf + j * BUF, o.in0, o.N, row0, o.M, col0 + 64 * j, o.N, lane);
          commit();
        }
      }
    } else if (K == DH) {
      block(p, o, buf, lane, row0, col0);
      block(p, o, buf + BUF, lane, row0, col0 + 32);
      sa = sb = 0;
      if (p.codes) {
        const uint8_t *s = p.scales + ((row0 + lane) * 2 * (int64_t)o.N + col0) / act8::kBlock;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const bool live = row0 + lane < o.M && 64 * j < o.width && col0 + 32 * j < o.N;
          sa |= (live ? (uint32_t)s[j] : 0u) << (8 * j);
          sb |= (live ? (uint32_t)s[j + o.N / act8::kBlock] : 0u) << (8 * j);
        }
      }
    }
  }
};

// a becomes act(a) b
template <bool CUBIC> __device__ __forceinline__ void gate16(float *a, const float *b, const Gate &g) {
#pragma unroll
  for (int i = 0; i < 16; i += 2)
    split(mul(ffn::gated2<CUBIC>(pair(a[i], a[i + 1]), g), pair(b[i], b[i + 1])), a[i], a[i + 1]);
}
// a becomes da = v b act'(a), v (dh) becomes db = v act(a), b becomes h = act(a) b
template <bool CUBIC> __device__ __forceinline__ void back16(float *a, float *b, float *v, const Gate &g) {
#pragma unroll
  for (int i = 0; i < 16; i += 2) {
    F2 act, slope;
    ffn::gate_and_slope2<CUBIC>(pair(a[i], a[i + 1]), g, act, slope);
    const F2 B = pair(b[i], b[i + 1]), V = pair(v[i], v[i + 1]);
    split(mul(mul(V, B), slope), a[i], a[i + 1]);
    split(mul(V, act), v[i], v[i + 1]);
    split(mul(B, act), b[i], b[i + 1]);
  }
}

// What becomes of the warp's slice: rows row0 .. row0 + 31 (a lane each), width / 2 columns from col0 on (GATEUP: width / 4
// features). Sixteen columns at a time in loops that stay loops: unrolled, most of the time of a first (or only) tile went into
// fetching the code.
template <int K>
__device__ __forceinline__ void finish(const Slice<K> &acc, Ahead<K> &ahead, const Params &p, const Product &o, uint32_t buf, int lane,
                                       int row0, int col0) {
  if (K == GATEUP) {
    const int row = row0 + lane, blocks = o.width / 128, end = min(o.N, col0 + 32 * blocks);
    const int64_t ld = 2 * (int64_t)o.N;
    if (p.codes) {
#pragma unroll 1
      for (int j = 0; j < blocks; ++j) {
        const int col = col0 + 32 * j;
        if (col >= o.N) break;
        float a[32], b[32];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          acc.load(32 * j + 16 * h, a + 16 * h);
          acc.load(acc.apart + 32 * j + 16 * h, b + 16 * h);
        }
        if (row < o.M) {
          uint8_t *c = p.codes + row * ld + col, *s = p.scales + (row * ld + col) / act8::kBlock;
          put_block8(c, s, a);
          put_block8(c + o.N, s + o.N / act8::kBlock, b);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (p.gate.k1 == 0.0f) gate16<false>(a + 16 * h, b + 16 * h, p.gate);
          else gate16<true>(a + 16 * h, b + 16 * h, p.gate);
        }
        stage<64, 4>(buf, lane, 4 * j, a);
      }
      if (col0 < o.N) put<64>(buf, lane, o.out1, o.N, row0, o.M, col0, end);
      return;
    }
    if (col0 >= o.N) return;
    // a and b leave through the two halves of the buffers (32 features each), h through the place of a
#pragma unroll 1
    for (int j = 0; j < blocks; ++j) {
      const int col = col0 + 32 * j;
      uint4 qh[4];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float a[16], b[16];
        acc.load(32 * j + 16 * h, a);
        acc.load(acc.apart + 32 * j + 16 * h, b);
        if (o.out0) {
          stage<32, 2>(buf, lane, 2 * h, a);
          stage<32, 2>(buf + 2048, lane, 2 * h, b);
        }
        if (p.gate.k1 == 0.0f) gate16<false>(a, b, p.gate);
        else gate16<true>(a, b, p.gate);
        qh[2 * h] = pack_bf16x8(a);
        qh[2 * h + 1] = pack_bf16x8(a + 8);
      }
      if (o.out0) {
        put<32>(buf, lane, o.out0, ld, row0, o.M, col, o.N);
        put<32>(buf + 2048, lane, o.out0 + o.N, ld, row0, o.M, col, o.N);
      }
#pragma unroll
      for (int c = 0; c < 4; ++c) st_shared_v4(Chunk<64>::at(buf + BUF, lane, 4 * j + c), qh[c]);
    }
    put<64>(buf + BUF, lane, o.out1, o.N, row0, o.M, col0, end);
  } else if (K == DH) {
    const int blocks = o.width / 64;
#pragma unroll 1
    for (int j = 0; j < blocks; ++j) {
      const int col = col0 + 32 * j;
      const uint32_t here = buf + (j & 1) * BUF;
      const int64_t ld = 2 * (int64_t)o.N;
      landed<1>();                    // the next block may be on its way
      if (col < o.N) {
        uint4 ca[2], cb[2], qh[4];
        if (p.codes) {   // before the buffer takes what is made of them
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            ca[h] = ld_shared_v4(code_at(here, lane, h));
            cb[h] = ld_shared_v4(code_at(here + 1024, lane, h));
          }
          __syncwarp();
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float a[16], b[16], v[16];
          acc.load(32 * j + 16 * h, v);
          if (p.codes) {
            unpack_codes(ca[h], act8::scale_value((ahead.sa >> (8 * j)) & 255u), a);
            unpack_codes(cb[h], act8::scale_value((ahead.sb >> (8 * j)) & 255u), b);
          } else {       // a lane's row of the buffer is its own: read, then overwritten
            take<32, 2, false>(here, lane, 2 * h, a);
            take<32, 2, false>(here + 2048, lane, 2 * h, b);
          }
          if (p.gate.k1 == 0.0f) back16<false>(a, b, v, p.gate);
          else back16<true>(a, b, v, p.gate);
          stage<32, 2>(here, lane, 2 * h, a);
          stage<32, 2>(here + 2048, lane, 2 * h, v);
          qh[2 * h] = pack_bf16x8(b);
          qh[2 * h + 1] = pack_bf16x8(b + 8);
        }
        put<32>(here, lane, o.out0, ld, row0, o.M, col, o.N);
        put<32>(here + 2048, lane, o.out0 + o.N, ld, row0, o.M, col, o.N);
        if (p.codes) {
#pragma unroll
          for (int c = 0; c < 4; ++c) st_shared_v4(Chunk<32>::at(here, lane, c), qh[c]);
          put<32>(here, lane, o.out1, o.N, row0, o.M, col, o.N);
        }
      }
      if (j + 2 < blocks) Ahead<K>::block(p, o, here, lane, row0, col + 64);
      else commit();                  // one group per block, for the count
    }
  } else {
    const bool add = o.in0 != nullptr;
#pragma unroll 1
    for (int j = 0; 128 * j < o.width; ++j) {
      const int col = col0 + 64 * j;
      const uint32_t here = buf + j * BUF;
      if (add) {
        if (j == 0) landed<1>();
        else landed<0>();
      }
      if (col >= o.N) continue;
#pragma unroll 1
      for (int h = 0; h < 4; h += 2) {   // a lane's row of the buffer is its own: read, then overwritten
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          float v[16];
          acc.load(64 * j + 16 * (h + g), v);
          if (add) take<64, 2, true>(here, lane, 2 * (h + g), v);
          stage<64, 2>(here, lane, 2 * (h + g), v);
        }
      }
      put<64>(here, lane, o.out0, o.N, row0, o.M, col, o.N);
    }
  }
}

// ---- tiles cut along K
// A warp's columns of its part, and what of the sum it finishes: the S warps that hold the parts of the same outputs share them
// in granules of 16 columns (GATEUP: 16 features, 32 where whole blocks are kept in 8 bits; DH: 16 columns), granule g is
// part g mod S's. All of it goes straight between registers and memory: it is little.
__device__ __forceinline__ float4 *part_of(const Params &p, const Product &o, int tile, int part, int slice, int c, int lane) {
  return p.part + ((int64_t)(o.at + tile * o.splits + part) * SLICES + slice) * (SLICE_FLOATS / 4) + (c / 4) * 32 + lane;
}
__device__ __forceinline__ void sum_parts(const Params &p, const Product &o, int tile, int slice, int c, int lane, float *v) {   // 16 columns from c on
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = 0.0f;
  const float4 *src = part_of(p, o, tile, 0, slice, c, lane);
  constexpr int64_t next = (int64_t)SLICES * SLICE_FLOATS / 4;
#pragma unroll 1
  for (int k = 0; k < o.splits; k += 4, src += 4 * next) {   // always in the parts' order, four parts' loads in flight
    float4 w[4][4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
#pragma unroll
      for (int i = 0; i < 4; ++i) w[u][i] = k + u < o.splits ? __ldcg(src + u * next + i * 32) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[4 * i] += w[u][i].x;
        v[4 * i + 1] += w[u][i].y;
        v[4 * i + 2] += w[u][i].z;
        v[4 * i + 3] += w[u][i].w;
      }
    }
  }
}
__device__ __forceinline__ void put16(__nv_bfloat16 *at, int col, int cols, const float *v) {
  if (col < cols) *reinterpret_cast<uint4 *>(at) = pack_bf16x8(v);
  if (col + 8 < cols) *reinterpret_cast<uint4 *>(at + 8) = pack_bf16x8(v + 8);
}
__device__ __forceinline__ void get16(const __nv_bfloat16 *at, int col, int cols, float *v) {
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = 0.0f;
  if (col < cols) unpack_bf16x8(*reinterpret_cast<const uint4 *>(at), v);
  if (col + 8 < cols) unpack_bf16x8(*reinterpret_cast<const uint4 *>(at + 8), v + 8);
}
template <int K>
__device__ __forceinline__ void finish_part(const Params &p, const Product &o, const Unit &t, int slice, int lane, int row, int col0) {
  const bool live = row < o.M;
  const int64_t at1 = (int64_t)row * o.N, at2 = 2 * at1;   // the row in [., N] and in [., 2 N]
  if (K == GATEUP && p.codes) {
#pragma unroll 1
    for (int g = t.part; g < o.width / 128; g += o.splits) {
      const int col = col0 + 32 * g;
      float a[32], b[32];
      if (col >= o.N) break;
#pragma unroll
      for (int h = 0; h < 32; h += 16) {
        sum_parts(p, o, t.tile, slice, 32 * g + h, lane, a + h);
        sum_parts(p, o, t.tile, slice, 64 + 32 * g + h, lane, b + h);
      }
      if (!live) continue;
      uint8_t *s = p.scales + (at2 + col) / act8::kBlock;
      put_block8(p.codes + at2 + col, s, a);
      put_block8(p.codes + at2 + o.N + col, s + o.N / act8::kBlock, b);
#pragma unroll
      for (int h = 0; h < 32; h += 16) {
        gate16<true>(a + h, b + h, p.gate);
        put16(o.out1 + at1 + col + h, col + h, o.N, a + h);
      }
    }
    return;
  }
#pragma unroll 1
  for (int g = t.part; g < o.width / (K == GATEUP ? 64 : 32); g += o.splits) {
    const int col = col0 + 16 * g;
    if (col >= o.N) break;
    float v[16];
    sum_parts(p, o, t.tile, slice, 16 * g, lane, v);
    if (K == GATEUP) {
      float b[16];
      sum_parts(p, o, t.tile, slice, 64 + 16 * g, lane, b);
      if (!live) continue;
      if (o.out0) {
        put16(o.out0 + at2 + col, col, o.N, v);
        put16(o.out0 + at2 + o.N + col, col, o.N, b);
      }
      gate16<true>(v, b, p.gate);
      put16(o.out1 + at1 + col, col, o.N, v);
    } else if (K == DH) {
      if (!live) continue;
      float a[16], b[16];
      if (p.codes) {
        const uint8_t *s = p.scales + (at2 + col) / act8::kBlock;
        unpack_codes(*reinterpret_cast<const uint4 *>(p.codes + at2 + col), act8::scale_value(s[0]), a);
        unpack_codes(*reinterpret_cast<const uint4 *>(p.codes + at2 + o.N + col), act8::scale_value(s[o.N / act8::kBlock]), b);
      } else {
        get16(o.in0 + at2 + col, col, o.N, a);
        get16(o.in0 + at2 + o.N + col, col, o.N, b);
      }
      back16<true>(a, b, v, p.gate);
      put16(o.out0 + at2 + col, col, o.N, a);
      put16(o.out0 + at2 + o.N + col, col, o.N, v);
      if (p.codes) put16(o.out1 + at1 + col, col, o.N, b);
    } else {
      if (!live) continue;
      if (o.in0) {
        float w[16];
        get16(o.in0 + at1 + col, col, o.N, w);
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] += w[i];
      }
      put16(o.out0 + at1 + col, col, o.N, v);
    }
  }
}

template <int CH>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(THREADS, 1)
    ffn_gemm_kernel(const __grid_constant__ Maps<CH> maps, const __grid_constant__ Params p) {
  constexpr bool B_MN = CH == BWD;
  auto a_mn = [&](const Unit &t) { return CH == BWD && p.prod[t.q].op == DW; };
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t *epi_smem = smem + STAGES * STAGE;
  uint64_t *bars = reinterpret_cast<uint64_t *>(epi_smem + EPI_WARPS * 2 * BUF);
  // bars: full[STAGES], empty[STAGES], tfull[2], tempty[2], mma_done
  uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(bars + NBARS);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_holder + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const uint32_t sbase = smem_u32(smem), bar0 = smem_u32(bars);
  auto full_bar = [&](int s) { return bar0 + 8u * s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (STAGES + s); };
  auto tfull_bar = [&](int a) { return bar0 + 8u * (2 * STAGES + a); };
  auto tempty_bar = [&](int a) { return bar0 + 8u * (2 * STAGES + 2 + a); };
  const uint32_t mma_done_bar = bar0 + 8u * (2 * STAGES + 4);

  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  Walk walk(pair, pairs, p);
  Unit t{};
  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(tfull_bar(a), 1);
      mbar_init(tempty_bar(a), 2 * EPI_WARPS);   // one arrival per epilogue warp of both CTAs
    }
    mbar_init(mma_done_bar, 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    for (int q = 0; q < products<CH>(); ++q) {
      asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&maps.a[q])) : "memory");
      asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&maps.b[q])) : "memory");
    }
  }
  if (warp == 1) {   // collective TMEM allocation by one warp of each CTA of the pair
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_holder)), "r"(2 * TILE)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  cluster_sync();   // both CTAs: barriers initialised, TMEM allocated
  tc_fence_after();
  const uint32_t tmem_base = *tmem_holder;
  bool more = walk.next(t, p);

  if (warp == 0) {
    // ------------------------------------------------------------------ TMA producer (both CTAs)
    // The whole warp runs the loop and waits, converged; one elected lane issues the copies.
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true, seen = false;      // seen: what the unit reads is known to be written
    Rows rows;
    while (ok && more) {
      const CUtensorMap *tmA = &maps.a[t.q], *tmB = &maps.b[t.q];
      const Product &o = p.prod[t.q];
      const bool along_m = a_mn(t);
      const int arow = t.m * TILE + (int)rank * HALF;
      const int half = o.width / 2, b_bytes = half * (BK * 2);
      const int brow = CH == FWD && o.op == GATEUP ? (int)rank * o.N + t.n * half : t.n * o.width + (int)rank * half;
      if (!seen && !rows.wait(p, o, t.m, abort_flag)) break;
      Unit nx{};
      more = walk.next(nx, p);
      seen = false;
      for (int kb = t.kb0; kb < t.kb1; ++kb) {
        // a look ahead for the next unit while this one's copies are still queued up
        if (kb == max(t.kb0, t.kb1 - 3)) seen = more && rows.look(p, p.prod[nx.q], nx.m);
        if (!spin_warp(empty_bar(stage), phase ^ 1u, abort_flag, p.hdr, 41)) {
          ok = false;
          break;
        }
        if (elect_one()) {
          const uint32_t sA = sbase + stage * STAGE, sB = sA + OPERAND;
          const uint32_t fb = mapa_shared(full_bar(stage), 0);   // the leader's full barrier
          if (leader) mbar_expect_tx(full_bar(stage), 2 * (OPERAND + b_bytes));
          const int kx = kb * BK;
          if (along_m) {
#pragma unroll
            for (int q = 0; q < 2; ++q) tma_load_2d_pair(sA + q * (BK * 128), tmA, arow + 64 * q, kx, fb);
          } else {
            tma_load_2d_pair(sA, tmA, kx, arow, fb);
          }
          if (B_MN) {
            for (int q = 0; 64 * q < half; ++q) tma_load_2d_pair(sB + q * (BK * 128), tmB, brow + 64 * q, kx, fb);
          } else {
            tma_load_2d_pair(sB, tmB, kx, brow, fb);
          }
        }
        __syncwarp();
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
      t = nx;
    }
  } else if (warp == 1 && leader) {
    // ------------------------------------------------------------------ MMA issuer (leader only)
    // Descriptors are formed once: every shared address lies below 256 KB, so a stage's or a k step's offset adds to the
    // start-address field without carry. K-major: 32 B per 16-deep step; MN-major: 2048 B per 16 k rows, the two
    // 64-wide blocks BK * 128 B apart.
    int stage = 0, acc = 0;
    uint32_t phase = 0, acc_phase = 0;
    bool ok = true, issued = false;
    const uint64_t desc_a_mn = sdesc(sbase, BK * 128, 1024), desc_a_k = sdesc(sbase, 16, 1024);
    const uint64_t desc_b = B_MN ? sdesc(sbase + OPERAND, BK * 128, 1024) : sdesc(sbase + OPERAND, 16, 1024);
    for (; ok && more; more = walk.next(t, p)) {
      const uint64_t desc_a = a_mn(t) ? desc_a_mn : desc_a_k;
      const uint32_t id = idesc(a_mn(t), B_MN, p.prod[t.q].width), a_step = a_mn(t) ? 2048 >> 4 : 32 >> 4;
      if (!wait_warp(tempty_bar(acc), acc_phase ^ 1u, abort_flag, p.hdr, 42)) break;
      tc_fence_after();
      const uint32_t d_tmem = tmem_base + (uint32_t)(acc * TILE);
      for (int kb = t.kb0; kb < t.kb1; ++kb) {
        if (!spin_warp(full_bar(stage), phase, abort_flag, p.hdr, 43)) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (elect_one()) {
          const uint32_t so = (uint32_t)(stage * STAGE) >> 4;
#pragma unroll
          for (int kk = 0; kk < BK / 16; ++kk)
            mma_bf16_pair(d_tmem, desc_a + so + (uint32_t)kk * a_step, desc_b + so + ((uint32_t)(kk * (B_MN ? 2048 : 32)) >> 4), id,
                          kb > t.kb0 || kk > 0 ? 1u : 0u);
          mma_commit_pair(empty_bar(stage), 0x3);   // frees this stage in both CTAs
        }
        __syncwarp();
        issued = true;
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
      if (!ok) break;
      if (elect_one()) mma_commit_pair(tfull_bar(acc), 0x3);   // both CTAs' accumulators are ready
      __syncwarp();
      acc ^= 1;
      if (acc == 0) acc_phase ^= 1u;
    }
    if (issued) {   // every MMA must have completed before TMEM is released
      if (elect_one()) mma_commit_pair(mma_done_bar, 0x1);
      __syncwarp();
      const uint64_t t0 = global_ns();
      while (!mbar_try_wait(mma_done_bar, 0) && global_ns() - t0 < kWaitLimitNs) {}
    }
  } else if (warp >= 2) {
    // ------------------------------------------------------------------ epilogue (both CTAs)
    const int quarter = warp & 3;                 // TMEM lanes 32 quarter .. 32 quarter + 31
    const int hh = (warp - 2) >> 2;               // which half of the columns
    const uint32_t buf = smem_u32(epi_smem) + (uint32_t)(warp - 2) * (2 * BUF);
    const int slice = (int)rank * EPI_WARPS + (warp - 2);
    int acc = 0;
    uint32_t acc_phase = 0;
    bool ok = true;
    // One unit of product `op`
    auto unit = [&](auto op) {
      constexpr int K = decltype(op)::value;
      const Product &o = p.prod[t.q];
      const int row0 = t.m * TILE + (int)rank * HALF + quarter * 32;
      const int mine = o.width / (K == GATEUP ? 4 : 2);   // columns (GATEUP: features) of this warp
      const int col0 = (2 * t.n + hh) * mine;
      const bool cut = t.part >= 0;
      Ahead<K> ahead;
      if (!cut) ahead.start(p, o, buf, lane, row0, col0);
      if (!wait_warp(tfull_bar(acc), acc_phase, abort_flag, p.hdr, 44)) return false;
      tc_fence_after();
      Slice<K> s;
      s.tmem = tmem_base + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(acc * TILE + mine * hh);
      s.apart = o.width / 2;
      if (cut) {
        float4 *out = part_of(p, o, t.tile, t.part, slice, 0, lane);
#pragma unroll 1
        for (int c = 0; c < o.width / 2; c += 16) {
          float v[16];
          s.load(K == GATEUP && c >= mine ? c - mine + s.apart : c, v);
          const int to = K == GATEUP && c >= mine ? c - mine + 64 : c;   // b's columns from 64 on
#pragma unroll
          for (int i = 0; i < 4; ++i) __stcg(out + (to / 4 + i) * 32, make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]));
        }
      } else {
        finish<K>(s, ahead, p, o, buf, lane, row0, col0);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive_leader(tempty_bar(acc));
      if (cut) {
        // the other parts' warps bring theirs without waiting for anything after this tile
        int *written = p.arrived + ((o.at + t.tile * o.splits) * SLICES + slice) * 2;
        __syncwarp();        // the other lanes' parts are visible before the count
        if (lane == 0) asm volatile("red.release.gpu.global.add.s32 [%0], 1;" ::"l"(written) : "memory");
        if (!wait_count(written, o.splits, abort_flag, p.hdr)) return false;
        finish_part<K>(p, o, t, slice, lane, row0 + lane, col0);
      }
      if (K == GATEUP || K == DH) {   // others in this launch read what this warp has written, by TMA
        asm volatile("fence.proxy.async.global;" ::: "memory");
        __syncwarp();
        if (lane == 0) asm volatile("red.release.gpu.global.add.s32 [%0], 1;" ::"l"(p.ready + t.m) : "memory");
      }
      if (cut) {
        int *written = p.arrived + ((o.at + t.tile * o.splits) * SLICES + slice) * 2, *left = written + 1;
        if (lane == 0 && atomicAdd(left, 1) == o.splits - 1) *written = *left = 0;
      }
      acc ^= 1;
      if (acc == 0) acc_phase ^= 1u;
      return true;
    };
    for (; ok && more; more = walk.next(t, p)) {
      const int op = p.prod[t.q].op;
      if (CH == FWD) {
        ok = op == GATEUP ? unit(std::integral_constant<int, GATEUP>()) : unit(std::integral_constant<int, DOWN>());
      } else {
        ok = op == DH ? unit(std::integral_constant<int, DH>()) : unit(std::integral_constant<int, DX>());
      }
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
  }

  if (*abort_flag) {   // copies that were issued and never waited for land within microseconds
    const uint64_t t0 = global_ns();
    while (global_ns() - t0 < 1000ull * 1000ull) {}
  }
  tc_fence_before();
  cluster_sync();   // no CTA leaves while its peer may still signal its barriers or use its TMEM
  if (leader && warp == 0) {   // nobody of this pair waits any more: the last pair clears up
    int before = 0;
    if (lane == 0) before = atomicAdd(p.left, 1);
    if (__shfl_sync(0xffffffffu, before, 0) == pairs - 1) {
      for (int r = lane; r < p.rows; r += 32) p.ready[r] = 0;
      if (lane == 0) *p.left = 0;
    }
  }
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(2 * TILE) : "memory");
  }
}

// ----------------------------------------------------------------------------- host side -------
// How a product is cut up: tiles of 256 or 128 columns, and along K. The costs are in units of 0.065 us, as measured at 389 x
// 2048 x 1024 and 256 x 4096 x 2048: a k-block takes 0.26 us at 256 columns and 0.19 at 128 (the copies bound both), the last
// epilogue 2-3 us or 1.2; a part, that leaves its fp32 accumulators, waits for the others' and adds up its share of them, 5.6 or
// 4.
struct Plan {
  int width, splits;
};
constexpr int kPartBlocks = 24;   // k-blocks that take as long as a part's exchange, about
constexpr int kBlockCost[2] = {4, 3}, kTileCost[2] = {38, 18}, kPartCost[2] = {48, 44};   // of 256 columns, of 128
static int64_t up(int64_t n, int64_t k) { return (n + k - 1) / k; }
static Plan plan(int64_t m_tiles, int64_t columns, int num_kb, int pairs) {
  Plan best{TILE, 1};
  int64_t least = INT64_MAX;
  for (int i = 0; i < 2; ++i) {
    const int64_t tiles = m_tiles * up(columns, TILE >> i);
    const int64_t per = num_kb * kBlockCost[i];
    // whole tiles: with more than one round the epilogues run beside the products
    const int64_t cost = up(tiles, pairs) * per + kTileCost[i];
    if (cost < least) {
      least = cost;
      best = {TILE >> i, 1};
    }
    if (tiles >= pairs) continue;   // with the call's other products in the same launch an incomplete round is evened out
    for (int s = 2; s <= MAX_SPLIT && s <= num_kb && tiles * s <= pairs; ++s) {
      const int64_t c = up(tiles * s, pairs) * (up(num_kb, s) * kBlockCost[i] + kTileCost[i] + kPartCost[i]);
      if (c < least) {
        least = c;
        best = {TILE >> i, s};
      }
    }
  }
  return best;
}
// The pairs that the plan counts on: those of a GB300, wherever it is asked for (the workspace's size follows from it).
constexpr int kPairs = 76;
constexpr int kPlaces = PRODUCTS * kPairs;   // of parts: every product may be cut, into kPairs parts at most
constexpr size_t kArrivedBytes = (size_t)kPlaces * SLICES * 8;
constexpr size_t kPartBytes = (size_t)SLICES * SLICE_FLOATS * 4;

template <auto KERNEL> static int pairs_resident(int &pairs) {
  static std::atomic<int> known[64];
  int dev = 0;
  MOE_TRY_CUDA(cudaGetDevice(&dev));
  if (dev < 64 && (pairs = known[dev].load(std::memory_order_relaxed)) > 0) return MOE_OK;
  MOE_TRY_CUDA(cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(sm_count() / 2 * 2), 1, 1);
  cfg.blockDim = dim3(THREADS, 1, 1);
  cfg.dynamicSmemBytes = SMEM;
  if (cudaOccupancyMaxActiveClusters(&pairs, KERNEL, &cfg) != cudaSuccess || pairs < 1) {
    (void)cudaGetLastError();
    pairs = sm_count() / 2;
  }
  if (dev < 64) known[dev].store(pairs, std::memory_order_relaxed);
  return MOE_OK;
}

// The counters in front of the parts: for cut tiles, then pairs that are done (one line), then rows of tiles. As many of these
// as the largest T has, whatever this call's is: a workspace may serve calls of any T, and parts never lie where another call
// counts on zeros.
constexpr size_t kReadyBytes = (MOE_FFN_MAX_T + TILE - 1) / TILE * sizeof(int);
constexpr size_t kCounterBytes = kArrivedBytes + 128 + kReadyBytes;
static_assert(kCounterBytes % 128 == 0, "parts start on a line");

// How the products' tiles are dealt to the pairs, product after product (in p.deal's order): parts of cut tiles in turn, whole
// tiles each to the pair with the least work so far (whole rounds at once, but for the last two). What waits for a first product
// of one round waits for all of it.
static void deal_out(Params &p, int pairs) {
  int64_t load[MAX_PAIRS] = {};
  memset(p.count, 0, sizeof(p.count));
  typedef std::pair<int64_t, int> Pair;   // a pair's work, and its number
  int next = 0, at = 0;
  for (int i = 0; i < p.products; ++i) {
    const int c = p.deal[i], wide = p.prod[c].width == TILE ? 0 : 1;
    Product &o = p.prod[c];
    int64_t n = (int64_t)o.m_tiles * o.n_tiles * o.splits;
    const int64_t cost = o.num_kb * kBlockCost[wide] / o.splits + (o.splits > 1 ? kTileCost[wide] + kPartCost[wide] : 8);
    if (o.splits > 1) {
      o.first = next;
      o.at = at;
      for (int64_t u = 0; u < n; ++u) load[(next + u) % pairs] += cost;
      next = (int)((next + n) % pairs);
      at += (int)n;
    } else {
      // A tile's cost is the same for all, so the pairs that have just got one come back in the order in which they got it: the least
      // work is at the front of the sorted pairs or of those.
      const int64_t even = n / pairs > 2 ? n / pairs - 2 : 0;
      Pair sorted[MAX_PAIRS], again[3 * MAX_PAIRS];
      for (int k = 0; k < pairs; ++k) {
        p.count[c][k] = (uint16_t)even;
        load[k] += even * cost;
        sorted[k] = {load[k], k};
      }
      std::sort(sorted, sorted + pairs);
      int front = 0, old = 0, last = 0;
      for (n -= even * pairs; n > 0; --n) {
        const Pair least = old < last && (front == pairs || again[old] < sorted[front]) ? again[old++] : sorted[front++];
        ++p.count[c][least.second];
        load[least.second] += cost;
        again[last++] = {load[least.second], least.second};
      }
    }
    if (i == 0 && (int64_t)o.m_tiles * o.n_tiles * o.splits <= pairs) {
      const int64_t most = *std::max_element(load, load + pairs);
      for (int k = 0; k < pairs; ++k) load[k] = most;
    }
  }
}

// Units wait for others of the same launch, so all its pairs have to be resident: a cooperative launch.
template <int CH> static int start(const Maps<CH> &maps, Params &p, const ffn::Block &blk, cudaStream_t s) {
  p.hdr = blk.hdr;
  p.gate = blk.gate;
  uint8_t *ws = (uint8_t *)blk.ws;
  p.arrived = (int *)ws;
  p.left = (int *)(ws + kArrivedBytes);
  p.ready = (int *)(ws + kArrivedBytes + 128);
  p.part = (float4 *)(ws + kCounterBytes);
  p.rows = p.prod[0].m_tiles;
  int pairs = 0;
  const int rc = pairs_resident<ffn_gemm_kernel<CH>>(pairs);
  if (rc) return rc;
  if (pairs > MAX_PAIRS) pairs = MAX_PAIRS;
  int64_t units = 0;
  for (int q = 0; q < p.products; ++q) {
    Product &o = p.prod[q];
    if (o.splits > pairs) o.splits = 1;   // the parts of a tile wait for one another: on as many pairs
    units += (int64_t)o.m_tiles * o.n_tiles * o.splits;
  }
  p.row_need = p.prod[0].n_tiles * SLICES * p.prod[0].splits;
  if (units > (int64_t)pairs * 60000) return MOE_ERR_UNSUPPORTED;   // counts have 16 bits
  if (pairs > units) pairs = (int)units;
  deal_out(p, pairs);
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeCooperative;
  attr.val.cooperative = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(2 * pairs);
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = SMEM;
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  MOE_TRY_CUDA(cudaLaunchKernelEx(&cfg, ffn_gemm_kernel<CH>, maps, p));
  return MOE_OK;
}

// One product; width 0: planned by itself
static Product product(int op, int64_t M, int64_t N, int64_t k, int width = 0) {
  Product o{};
  o.op = op;
  o.M = (int)M;
  o.N = (int)N;
  o.m_tiles = (int)up(M, TILE);
  o.num_kb = (int)up(k, BK);
  const int64_t columns = op == GATEUP ? 2 * N : N;
  const Plan how = width ? Plan{width, 1} : plan(o.m_tiles, columns, o.num_kb, kPairs);
  o.width = how.width;
  o.splits = how.splits;
  o.n_tiles = (int)up(columns, o.width);
  return o;
}
static size_t part_bytes(const Product &o) { return o.splits > 1 ? (size_t)o.m_tiles * o.n_tiles * o.splits * kPartBytes : 0; }

// The backward's products. The last three run beside one another: narrow tiles where they give every pair one at most, and a product
// whose K takes a tile much longer than a pair's share of all three (or, less than that, than a part costs) is cut along it:
// 101 to 52 us for a step of 234 x 72 x 6768, whose dx is one tile of 212 k-blocks.
struct Backward {
  Product dh, dx, down, gu;
};
static Backward backward_of(int64_t T, int64_t d, int64_t f) {
  const int64_t narrow = up(T, TILE) * up(d, HALF) + up(d, TILE) * up(f, HALF) + up(2 * f, TILE) * up(d, HALF);
  const int width = narrow <= kPairs ? HALF : TILE;
  Backward b{product(DH, T, f, d), product(DX, T, d, 2 * f, width), product(DW, d, f, T, width), product(DW, 2 * f, d, T, width)};
  Product *const three[3] = {&b.dx, &b.down, &b.gu};
  int64_t work = 0;
  for (const Product *o : three) work += (int64_t)o->m_tiles * o->n_tiles * o->num_kb;
  const int64_t share = std::max(work / kPairs, (int64_t)kPartBlocks);
  for (Product *o : three) {
    const int64_t tiles = (int64_t)o->m_tiles * o->n_tiles;
    if (tiles == 0 || 2 * o->num_kb <= 3 * share || tiles > kPairs) continue;   // (no tokens: dx has no tiles)
    o->splits = (int)std::min({up(o->num_kb, share), (int64_t)MAX_SPLIT, kPairs / tiles});
  }
  return b;
}
}  // namespace ffng
}  // namespace tc

namespace ffn {

using namespace tc;
using namespace tc::ffng;
typedef __nv_bfloat16 bf16;

size_t gemm_workspace(int T, int d, int f, bool backward) {
  size_t most = part_bytes(product(GATEUP, T, f, d)) + part_bytes(product(DOWN, T, d, f));
  if (backward) {
    const Backward b = backward_of(T, d, f);
    most = std::max(most, part_bytes(b.dh) + part_bytes(b.dx) + part_bytes(b.down) + part_bytes(b.gu));
  }
  return kCounterBytes + most;
}

// Forward: y's tiles wait for the rows of h that they read.
int gemm_fwd(const Block &b, cudaStream_t s) {
  Product up_ = product(GATEUP, b.T, b.f, b.d), down = product(DOWN, b.T, b.d, b.f);
  Maps<FWD> m;
  if (!make_map(&m.a[0], b.x, b.T, b.d, HALF) || !make_map(&m.b[0], b.w_gate_up, 2 * (uint64_t)b.f, b.d, up_.width / 2) ||
      !make_map(&m.a[1], b.h, b.T, b.f, HALF) || !make_map(&m.b[1], b.w_down, b.d, b.f, down.width / 2))
    return MOE_ERR_CUDA;
  Params p{};
  if (b.scales) {
    p.codes = (uint8_t *)b.ab;
    p.scales = b.scales;
  } else {
    up_.out0 = (bf16 *)b.ab;
  }
  up_.out1 = (bf16 *)b.h;
  down.in0 = (const bf16 *)b.add;
  down.out0 = (bf16 *)b.y;
  down.needs = ITS_ROWS;
  p.prod[0] = up_;
  p.prod[1] = down;
  p.products = 2;
  p.deal[1] = 1;
  return start<FWD>(m, p, b, s);
}

// Backward: da, db (and h, from 8 bits), then dx = dab Wgu (+ dx_in), dWd = dy^T h and dWgu = dab^T x, in one launch. dx waits
// for the rows of dab that it reads, which are there first, dWgu for all of them, dWd for nothing (for all rows of h where those
// are written here): it is taken first then, by the pairs that the first product leaves with the least work. The longer tiles
// are dealt out before the shorter ones, which even out what those leave.
int gemm_bwd(const Block &b, cudaStream_t s) {
  const uint64_t T = b.T, d = b.d, f = b.f;
  Backward products = backward_of(b.T, b.d, b.f);
  Product &dh = products.dh, &dx = products.dx, &down = products.down, &gu = products.gu;
  Params p{};
  if (b.scales) {
    p.codes = (uint8_t *)b.ab;
    p.scales = b.scales;
    dh.out1 = (bf16 *)b.h;
  } else {
    dh.in0 = (const bf16 *)b.ab;
  }
  dh.out0 = (bf16 *)b.dab;
  dx.in0 = (const bf16 *)b.add;
  dx.out0 = (bf16 *)b.dx;
  down.out0 = (bf16 *)b.dw_down;
  gu.out0 = (bf16 *)b.dw_gate_up;
  const bool dx_longer = dx.num_kb > gu.num_kb;
  dx.needs = ITS_ROWS;
  gu.needs = ALL_ROWS;
  down.needs = b.scales ? ALL_ROWS : NOTHING;
  const int ix = b.scales ? 1 : 2, iw = 3 - ix;   // dx and dWd
  Maps<BWD> m;
  p.prod[0] = dh;
  p.prod[ix] = dx;
  p.prod[iw] = down;
  p.prod[3] = gu;
  if (!make_map(&m.a[0], b.dy, T, d, HALF) || !make_map(&m.b[0], b.w_down, d, f, BK) || !make_map(&m.a[ix], b.dab, T, 2 * f, HALF) ||
      !make_map(&m.b[ix], b.w_gate_up, 2 * f, d, BK) || !make_map(&m.a[iw], b.dy, T, d, BK) || !make_map(&m.b[iw], b.h, T, f, BK) ||
      !make_map(&m.a[3], b.dab, T, 2 * f, BK) || !make_map(&m.b[3], b.x, T, d, BK))
    return MOE_ERR_CUDA;
  p.products = 4;
  p.deal[1] = dx_longer ? ix : iw;
  p.deal[2] = dx_longer ? iw : 3;
  p.deal[3] = dx_longer ? 3 : ix;
  return start<BWD>(m, p, b, s);
}

}  // namespace ffn
}  // namespace moe
