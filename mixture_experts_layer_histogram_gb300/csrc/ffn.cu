// C-ABI entry points of the gated feed-forward block: checks, then the path for the type and size.
#include "ffn.cuh"

using namespace moe;
using namespace moe::ffn;

static bool bad(const void *p) { return !p || !aligned16(p); }
constexpr size_t kHeader = 256;

static int check(int T, int d, int f, int dtype, int act, int keep) {
  if (T < 0 || d < 1 || f < 1 || (dtype != MOE_F32 && dtype != MOE_BF16) || (act != MOE_ACT_SILU && act != MOE_ACT_GELU) ||
      keep < MOE_KEEP_NONE || keep > MOE_KEEP_F8)
    return MOE_ERR_INVALID_ARG;
  if (d > MOE_FFN_MAX || f > MOE_FFN_MAX || T > MOE_FFN_MAX_T) return MOE_ERR_UNSUPPORTED;
  if (dtype == MOE_BF16 && (d % 8 || f % 8)) return MOE_ERR_UNSUPPORTED;
  if (keep == MOE_KEEP_F8 && (dtype != MOE_BF16 || f % act8::kBlock)) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// Few tokens: the path that reads the weights once, whose blocks each read all tokens. With more of those than 32 and large weights
// that reading costs more than the tiles of the other path. This one and the other, in us: 44 and 57 for 32 tokens of 4096 x
// 8192 (201 MB), 57 and 57 for 48, 77 and 57 for 64; for 48 of 8192 x 16384 (805 MB) 193 and 164; for 64 of 4096 x 2048 23 and 30,
// of 2048 x 8192 (101 MB) 39 and 39. Without its ring (few_ring), in replayed graphs: 16 tokens of 8200 x 16392 148 and 160, of 4104 x
// 8200 47 and 57; 32 of that 67 and 57, of 2056 x 8200 49 and 38, of 4104 x 4104 36 and 43, of 1000 x 10248 (61 MB) 36 and 38, of 2056
// x 5128 (63 MB) 35 and 31, of 4104 x 2056 (51 MB) 20 and 30; 48 of that 27 and 31, of 2056 x 4104 (51 MB) 35 and 28, of 8200 x 1032 36 and
// 33; 64 of 2056 x 2056 (25 MB) 21 and 24, of 1000 x 4104 29 and 24, of 1000 x 2056 16 and 19.
static bool few(int T, int d, int f) {
  const int64_t weights = (int64_t)6 * d * f, MiB = 1 << 20;
  if (few_ring(T, d, f)) return T <= 32 || (T <= 48 && weights <= 512 * MiB) || (T <= kFewTokens && weights <= 128 * MiB);
  return T <= 16 || (T <= 32 && weights <= 64 * MiB) || (T <= kFewTokens && weights <= 25 * MiB);
}

extern "C" size_t moe_ffn_workspace_size(int T, int d, int f, int dtype, int backward) {
  if (check(T, d, f, dtype, MOE_ACT_SILU, MOE_KEEP_NONE)) return 0;
  return kHeader + (dtype == MOE_BF16 ? gemm_workspace(T, d, f, backward != 0) : 0);
}

static int check_ws(const void *ws, size_t bytes, int T, int d, int f, int dtype, int backward) {
  return !ws || ((uintptr_t)ws & 255) || bytes < moe_ffn_workspace_size(T, d, f, dtype, backward) ? MOE_ERR_INVALID_ARG : MOE_OK;
}

extern "C" int moe_ffn_fwd(const void *x, const void *w_gate_up, const void *w_down, const void *y_in, int T, int d, int f,
                           int dtype, int act, int keep, void *ab, void *ab_scales, void *h, void *y, void *ws,
                           size_t ws_bytes, moe_stream_t stream) {
  int rc = check(T, d, f, dtype, act, keep);
  if (rc) return rc;
  if ((rc = check_ws(ws, ws_bytes, T, d, f, dtype, 0))) return rc;
  if ((ab != nullptr) != (keep != MOE_KEEP_NONE) || (ab_scales != nullptr) != (keep == MOE_KEEP_F8)) {
    if (T > 0) return MOE_ERR_INVALID_ARG;
  }
  if (T == 0) return MOE_OK;
  if (bad(x) || bad(w_gate_up) || bad(w_down) || bad(h) || bad(y) || !aligned16(y_in) || !aligned16(ab) || !aligned16(ab_scales))
    return MOE_ERR_INVALID_ARG;
  Block b{};
  b.T = T;
  b.d = d;
  b.f = f;
  b.gate = gate_of(act);
  b.x = x;
  b.w_gate_up = w_gate_up;
  b.w_down = w_down;
  b.add = y_in;
  b.ab = ab;
  b.scales = (uint8_t *)ab_scales;
  b.h = h;
  b.y = y;
  b.hdr = (WsHeader *)ws;
  b.ws = (uint8_t *)ws + kHeader;
  cudaStream_t s = (cudaStream_t)stream;
  if (dtype == MOE_F32) return f32_fwd(b, s);
  return keep == MOE_KEEP_NONE && few(T, d, f) ? few_fwd(b, s) : gemm_fwd(b, s);
}

extern "C" int moe_ffn_bwd(const void *dy, const void *x, const void *ab, const void *ab_scales, void *h, const void *w_gate_up,
                           const void *w_down, const void *dx_in, int T, int d, int f, int dtype, int act, int keep, void *dab,
                           void *dx, void *dw_gate_up, void *dw_down, void *ws, size_t ws_bytes, moe_stream_t stream) {
  int rc = check(T, d, f, dtype, act, keep);
  if (rc) return rc;
  if (keep == MOE_KEEP_NONE) return MOE_ERR_INVALID_ARG;
  if ((rc = check_ws(ws, ws_bytes, T, d, f, dtype, 1))) return rc;
  if (bad(dw_gate_up) || bad(dw_down)) return MOE_ERR_INVALID_ARG;
  cudaStream_t s = (cudaStream_t)stream;
  if (T == 0) {
    const size_t n = (size_t)d * f * dtype_size(dtype);
    MOE_TRY_CUDA(cudaMemsetAsync(dw_gate_up, 0, 2 * n, s));
    MOE_TRY_CUDA(cudaMemsetAsync(dw_down, 0, n, s));
    return MOE_OK;
  }
  if (bad(dy) || bad(x) || bad(ab) || bad(h) || bad(w_gate_up) || bad(w_down) || !aligned16(dx_in) || bad(dab) || bad(dx) ||
      (ab_scales != nullptr) != (keep == MOE_KEEP_F8) || !aligned16(ab_scales))
    return MOE_ERR_INVALID_ARG;
  Block b{};
  b.T = T;
  b.d = d;
  b.f = f;
  b.gate = gate_of(act);
  b.x = x;
  b.w_gate_up = w_gate_up;
  b.w_down = w_down;
  b.add = dx_in;
  b.ab = const_cast<void *>(ab);
  b.scales = (uint8_t *)const_cast<void *>(ab_scales);
  b.h = h;
  b.dy = dy;
  b.dab = dab;
  b.dx = dx;
  b.dw_gate_up = dw_gate_up;
  b.dw_down = dw_down;
  b.hdr = (WsHeader *)ws;
  b.ws = (uint8_t *)ws + kHeader;
  return dtype == MOE_F32 ? f32_bwd(b, s) : gemm_bwd(b, s);
}
