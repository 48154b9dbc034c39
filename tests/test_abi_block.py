"""Arguments that the norms, the optimiser step and the MXFP4 calls refuse on the host (no GPU needed)."""
import ctypes
import os

import pytest

FAKE = ctypes.c_void_p(1 << 20)   # never dereferenced: every call below fails validation first
ODD = ctypes.c_void_p((1 << 20) + 4)
NULL = None


@pytest.fixture(scope="module")
def L():
    from mixture_experts_layer_histogram_gb300 import _lib, build
    if not os.path.exists(_lib.LIB_PATH):
        build.build()
    return _lib.lib()


def test_norm_refusals(L):
    assert L.moe_norm_fwd(FAKE, FAKE, 4, 0, 0, 1e-6, FAKE, NULL) == -1
    assert L.moe_norm_fwd(FAKE, FAKE, -1, 64, 0, 1e-6, FAKE, NULL) == -1
    assert L.moe_norm_fwd(FAKE, FAKE, 4, 64, 2, 1e-6, FAKE, NULL) == -1
    assert L.moe_norm_fwd(FAKE, FAKE, 4, 64, 0, 0.0, FAKE, NULL) == -1
    assert L.moe_norm_fwd(FAKE, FAKE, 4, 64, 0, float("nan"), FAKE, NULL) == -1
    assert L.moe_norm_fwd(FAKE, FAKE, 4, 8193, 0, 1e-6, FAKE, NULL) == -2
    assert L.moe_norm_fwd(ODD, FAKE, 4, 64, 0, 1e-6, FAKE, NULL) == -1
    assert L.moe_norm_fwd(FAKE, NULL, 4, 64, 0, 1e-6, FAKE, NULL) == -1
    assert L.moe_norm_fwd(NULL, NULL, 0, 64, 0, 1e-6, NULL, NULL) == 0
    # gate kind, a missing gate, an n without w_next and the other way round
    assert L.moe_norm_residual_fwd(FAKE, FAKE, FAKE, FAKE, 3, NULL, 4, 64, 0, 1.0, 1e-6, FAKE, NULL, NULL) == -1
    assert L.moe_norm_residual_fwd(FAKE, FAKE, FAKE, NULL, 1, NULL, 4, 64, 0, 1.0, 1e-6, FAKE, NULL, NULL) == -1
    assert L.moe_norm_residual_fwd(FAKE, FAKE, FAKE, NULL, 0, NULL, 4, 64, 0, 1.0, 1e-6, FAKE, FAKE, NULL) == -1
    assert L.moe_norm_residual_fwd(FAKE, FAKE, FAKE, NULL, 0, FAKE, 4, 64, 0, 1.0, 1e-6, FAKE, NULL, NULL) == -1
    ws = L.moe_norm_bwd_workspace_size(4, 64, 0)
    assert ws >= 2 * 64 * 4
    assert L.moe_norm_bwd(FAKE, FAKE, FAKE, NULL, 4, 64, 0, 1e-6, FAKE, FAKE, FAKE, ws - 1, NULL) == -1
    assert L.moe_norm_bwd(FAKE, FAKE, FAKE, NULL, 4, 64, 0, 1e-6, FAKE, NULL, FAKE, ws, NULL) == -1
    assert L.moe_norm_bwd(FAKE, FAKE, FAKE, NULL, 4, 64, 0, 1e-6, FAKE, FAKE, ODD, ws, NULL) == -1
    res = L.moe_norm_residual_bwd
    # dn without w_next; neither dout nor dn; a gate without its gradient
    assert res(FAKE, FAKE, FAKE, FAKE, FAKE, NULL, 0, NULL, 4, 64, 0, 1.0, 1e-6, FAKE, FAKE, FAKE, NULL, NULL, FAKE, ws,
               NULL) == -1
    assert res(NULL, NULL, NULL, FAKE, FAKE, NULL, 0, NULL, 4, 64, 0, 1.0, 1e-6, FAKE, FAKE, FAKE, NULL, NULL, FAKE, ws,
               NULL) == -1
    assert res(FAKE, NULL, NULL, FAKE, FAKE, FAKE, 1, NULL, 4, 64, 0, 1.0, 1e-6, FAKE, FAKE, FAKE, NULL, NULL, FAKE, ws,
               NULL) == -1


def test_adamw_plans(L):
    from mixture_experts_layer_histogram_gb300 import _lib
    T = _lib.AdamWTensor

    def plan(**kw):
        a = T(**{**dict(p=4096, g=4096, m=4096, v=4096, n=10, dtype=0, state=0), **kw})
        size = L.moe_adamw_plan_size(ctypes.byref(a), 1)
        buf = (ctypes.c_int64 * (size // 8 + 1))()
        return L.moe_adamw_plan(ctypes.byref(a), 1, buf, size)

    assert plan() == 0
    assert plan(n=0, p=None, g=None, m=None, v=None) == 0
    assert plan(n=-1) == -1
    assert plan(p=None) == -1 and plan(g=None) == -1 and plan(m=None) == -1 and plan(v=None) == -1
    assert plan(p=4098) == -1 and plan(p=4098, g=4098, dtype=1) == 0
    assert plan(dtype=2) == -1 and plan(state=2) == -1
    assert plan(weight_decay=-0.1) == -1 and plan(weight_decay=float("nan")) == -1
    assert plan(master=4096) == -1 and plan(master=4096, dtype=1) == 0
    assert plan(state=1) == -1                                  # 8-bit states without scales
    assert plan(state=1, m_scale=4096, v_scale=4096) == 0
    with pytest.raises(_lib.MoeError):
        _lib._ok("moe_adamw_plan", L.moe_adamw_plan(None, 1, FAKE, 64))
    # a chunk of 4096 values is 8 bytes of the plan
    sizes = [L.moe_adamw_plan_size(ctypes.byref(T(n=n)), 1) for n in (0, 1, 4096, 4097, 1 << 30)]
    assert [s - sizes[0] for s in sizes] == [0, 8, 8, 16, 8 << 18]
    host = _lib.moe_adamw_plan([T(p=4096, g=4096, m=4096, v=4096, n=10)])
    ptr = ctypes.c_void_p(host.data_ptr())
    for args in ((NULL, FAKE, .9, .99, 1e-8, FAKE), (ptr, NULL, .9, .99, 1e-8, FAKE), (ptr, FAKE, 1.0, .99, 1e-8, FAKE),
                 (ptr, FAKE, .9, -.1, 1e-8, FAKE), (ptr, FAKE, .9, .99, 0.0, FAKE), (ptr, FAKE, .9, .99, 1e-8, NULL),
                 (ptr, ctypes.c_void_p((1 << 20) + 8), .9, .99, 1e-8, FAKE)):
        assert L.moe_adamw_step(*args, NULL) == -1
    host[0] = 0                                                 # no plan
    assert L.moe_adamw_step(ptr, FAKE, .9, .99, 1e-8, FAKE, NULL) == -1


def test_fp4_refusals(L):
    assert L.moe_fp4_scale_bytes(129, 160) == 2 * 2 * 512 and L.moe_fp4_scale_bytes(0, 32) == 0
    assert L.moe_fp4_quantize(FAKE, 1, 4, 48, FAKE, FAKE, NULL) == -2
    assert L.moe_fp4_quantize(FAKE, 2, 4, 64, FAKE, FAKE, NULL) == -1
    assert L.moe_fp4_quantize(FAKE, 1, -1, 64, FAKE, FAKE, NULL) == -1
    assert L.moe_fp4_quantize(ODD, 1, 4, 64, FAKE, FAKE, NULL) == -1
    assert L.moe_fp4_quantize(NULL, 1, 0, 64, NULL, NULL, NULL) == 0
    assert L.moe_fp4_dequantize(FAKE, NULL, 4, 64, 1, FAKE, NULL) == -1
    assert L.moe_fp4_dequantize(FAKE, FAKE, 4, 63, 1, FAKE, NULL) == -2
    rm = L.moe_grouped_rows_max(64, 2, 8)
    assert L.moe_permute_fp4(FAKE, 1, 64, 96, 2, 8, FAKE, FAKE, FAKE, rm, FAKE, FAKE, NULL) == -2
    assert L.moe_permute_fp4(FAKE, 1, 64, 128, 2, 8, FAKE, FAKE, FAKE, rm - 128, FAKE, FAKE, NULL) == -1
    assert L.moe_permute_fp4(FAKE, 1, 64, 128, 17, 8, FAKE, FAKE, FAKE, rm, FAKE, FAKE, NULL) == -1
    ws = L.moe_grouped_ffn_workspace_size(8, 256, 256, rm, 1, 0)

    def ffn(E=8, d=256, f=256, rows=rm, y=FAKE, w=FAKE, n=ws):
        return L.moe_grouped_ffn_fwd_fp4(FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, E, d, f, rows, FAKE, FAKE, y, w, n,
                                         NULL)
    assert ffn(d=128) == -2 and ffn(f=384) == -2 and ffn(E=0) == -1 and ffn(E=300) == -1
    assert ffn(rows=rm + 1) == -1 and ffn(y=NULL) == -1 and ffn(w=NULL) == -1 and ffn(n=8) == -1 and ffn(w=ODD) == -1
    assert ffn(rows=0) == 0


def test_norm_backward_without_rows_still_wants_its_weights(L):
    """The kernel reads w before its first row, so a missing w is refused with T = 0 as well."""
    ws = L.moe_norm_bwd_workspace_size(0, 64, 0)
    assert L.moe_norm_bwd(NULL, NULL, NULL, NULL, 0, 64, 0, 1e-6, NULL, FAKE, FAKE, ws, NULL) == -1
    assert L.moe_norm_bwd(NULL, NULL, ODD, NULL, 0, 64, 0, 1e-6, NULL, FAKE, FAKE, ws, NULL) == -1


def test_adamw_plan_of_too_many_values(L):
    from mixture_experts_layer_histogram_gb300 import _lib
    buf = (ctypes.c_int64 * 64)()
    for n in ((1 << 63) - 1, 1 << 43):
        a = _lib.AdamWTensor(p=4096, g=4096, m=4096, v=4096, n=n, dtype=0, state=0)
        assert L.moe_adamw_plan(ctypes.byref(a), 1, buf, ctypes.sizeof(buf)) == -2
