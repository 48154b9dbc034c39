"""Arguments that the gated feed-forward block refuses on the host (no GPU needed)."""
import ctypes
import os

import pytest
import torch

from test_abi_activations import B, Claimed   # noqa: F401  (a fixture)

FAKE = ctypes.c_void_p(1 << 20)   # never dereferenced: every call below fails validation first
ODD = ctypes.c_void_p((1 << 20) + 4)
NULL = None
F32, BF16 = 0, 1
NONE, ALL, F8 = 0, 1, 2


@pytest.fixture(scope="module")
def L():
    from mixture_experts_layer_histogram_gb300 import _lib, build
    if not os.path.exists(_lib.LIB_PATH):
        build.build()
    return _lib.lib()


def test_workspace_sizes(L):
    size = L.moe_ffn_workspace_size
    assert size(-1, 64, 64, 1, 0) == size(4, 0, 64, 1, 0) == size(4, 64, 64, 2, 0) == size(4, 60, 64, 1, 0) == 0
    assert size(4, 61, 63, F32, 1) >= 64
    for T in (1, 64, 65, 1000, 8192, 100000):
        assert 64 <= size(T, 2048, 1024, BF16, 0) <= size(T, 2048, 1024, BF16, 1) <= 64 << 20


def test_forward_refusals(L):
    ws = max(L.moe_ffn_workspace_size(70, 64, 64, t, 1) for t in (F32, BF16))

    def fwd(x=FAKE, wgu=FAKE, wd=FAKE, y_in=NULL, T=70, d=64, f=64, dtype=BF16, act=0, keep=NONE, ab=NULL, sc=NULL, h=FAKE, y=FAKE,
            w=FAKE, n=ws):
        return L.moe_ffn_fwd(x, wgu, wd, y_in, T, d, f, dtype, act, keep, ab, sc, h, y, w, n, NULL)

    for k in ("x", "wgu", "wd", "h", "y", "w"):
        assert fwd(**{k: NULL}) == fwd(**{k: ODD}) == -1, k
    assert fwd(y_in=ODD) == fwd(n=L.moe_ffn_workspace_size(70, 64, 64, BF16, 0) - 1) == fwd(w=ctypes.c_void_p((1 << 20) + 64)) == -1
    assert fwd(T=-1) == fwd(d=0) == fwd(f=0) == fwd(dtype=2) == fwd(act=2) == fwd(act=-1) == fwd(keep=3) == -1
    assert fwd(d=60) == fwd(f=60) == fwd(d=(1 << 20) + 8) == fwd(T=(1 << 22) + 1) == -2
    assert fwd(keep=F8, ab=FAKE, sc=FAKE, f=40) == fwd(keep=F8, ab=FAKE, sc=FAKE, dtype=F32) == -2
    # ab and scales given exactly where they are kept
    assert fwd(ab=FAKE) == fwd(sc=FAKE) == fwd(keep=ALL) == fwd(keep=ALL, ab=FAKE, sc=FAKE) == fwd(keep=F8, ab=FAKE) == fwd(keep=F8, sc=FAKE) == -1
    assert fwd(keep=ALL, ab=ODD) == fwd(keep=F8, ab=FAKE, sc=ODD) == -1
    assert fwd(T=0, x=NULL, wgu=NULL, h=NULL, y=NULL) == 0


def test_backward_refusals(L):
    ws = L.moe_ffn_workspace_size(70, 64, 64, BF16, 1)

    def bwd(dy=FAKE, x=FAKE, ab=FAKE, sc=NULL, h=FAKE, wgu=FAKE, wd=FAKE, dx_in=NULL, T=70, d=64, f=64, dtype=BF16, act=0, keep=ALL,
            dab=FAKE, dx=FAKE, dwgu=FAKE, dwd=FAKE, w=FAKE, n=ws):
        return L.moe_ffn_bwd(dy, x, ab, sc, h, wgu, wd, dx_in, T, d, f, dtype, act, keep, dab, dx, dwgu, dwd, w, n, NULL)

    for k in ("dy", "x", "ab", "h", "wgu", "wd", "dab", "dx", "dwgu", "dwd", "w"):
        assert bwd(**{k: NULL}) == bwd(**{k: ODD}) == -1, k
    assert bwd(dx_in=ODD) == bwd(n=ws - 1) == bwd(keep=NONE) == bwd(keep=F8) == bwd(sc=FAKE) == bwd(keep=F8, sc=ODD) == -1
    assert bwd(T=-1) == bwd(dtype=7) == bwd(act=5) == -1
    assert bwd(d=4) == bwd(keep=F8, sc=FAKE, f=8) == -2


def test_binding_refusals(B):   # noqa: F811
    L, calls = B
    bf, u8 = torch.bfloat16, torch.uint8
    T, d, f = 4, 64, 32
    n = Claimed
    fwd = dict(x=n(T, d, dtype=bf), w_gate_up=n(2 * f, d, dtype=bf), w_down=n(d, f, dtype=bf), y_in=n(T, d, dtype=bf), ab=n(T, 2 * f, dtype=u8),
               ab_scales=n(T * 2, dtype=u8), h=n(T, f, dtype=bf), y=n(T, d, dtype=bf), ws=n(64, dtype=u8))
    bwd = dict(dy=n(T, d, dtype=bf), x=n(T, d, dtype=bf), ab=n(T, 2 * f, dtype=u8), ab_scales=n(T * 2, dtype=u8), h=n(T, f, dtype=bf),
               w_gate_up=n(2 * f, d, dtype=bf), w_down=n(d, f, dtype=bf), dx_in=n(T, d, dtype=bf), dab=n(T, 2 * f, dtype=bf), dx=n(T, d, dtype=bf),
               dw_gate_up=n(2 * f, d, dtype=bf), dw_down=n(d, f, dtype=bf), ws=n(64, dtype=u8))
    L.moe_ffn_fwd(**fwd)
    L.moe_ffn_fwd(**{**fwd, "ab": None, "ab_scales": None, "y_in": None})
    L.moe_ffn_fwd(**{**fwd, "ab": n(T, 2 * f, dtype=bf), "ab_scales": None})
    L.moe_ffn_bwd(**bwd)
    assert [c[1][9] for c in calls[:3]] == [F8, NONE, ALL]
    for fn, args in ((L.moe_ffn_fwd, fwd), (L.moe_ffn_bwd, bwd)):
        for k, t in args.items():
            shape = tuple(t.shape)
            wrong = [n(*shape, dtype=t.dtype, device=1)]
            if k != "ws":
                wrong += [n(*shape, dtype=torch.float16), n(*(s - 1 for s in shape), dtype=t.dtype)]
                if len(shape) == 2:
                    strided = n(shape[0], 2 * shape[1], dtype=t.dtype)
                    strided._t = strided._t[:, ::2]
                    wrong.append(strided)
            for bad in wrong:
                with pytest.raises((ValueError, TypeError)):
                    fn(**{**args, k: bad})
    with pytest.raises(ValueError, match="ab_scales"):
        L.moe_ffn_fwd(**{**fwd, "ab": None})
    assert len(calls) == 4


def test_class_refusals():
    from mixture_experts_layer_histogram_gb300 import GatedFFN
    with pytest.raises(ValueError, match="act"):
        GatedFFN(4, 64, 64, act="relu")
    with pytest.raises(ValueError, match="keep"):
        GatedFFN(4, 64, 64, keep="f4")
    with pytest.raises(ValueError, match="backward"):
        GatedFFN(4, 64, 64, keep="f8", backward=False)
    ffn = GatedFFN.__new__(GatedFFN)
    ffn.backward_enabled = False
    with pytest.raises(RuntimeError, match="backward"):
        ffn.backward(None, None, None, None)


def test_another_current_gpu(monkeypatch):
    from mixture_experts_layer_histogram_gb300 import GatedFFN, LayerNorm
    from mixture_experts_layer_histogram_gb300 import _lib
    monkeypatch.setattr(_lib, "_device", lambda: 1)
    ffn, norm = GatedFFN.__new__(GatedFFN), LayerNorm.__new__(LayerNorm)
    ffn._index = norm._index = 0
    norm.bias = False
    with pytest.raises(ValueError, match="cuda:0"):
        ffn.forward(None, None, None)
    with pytest.raises(ValueError, match="cuda:0"):
        norm.forward(None, None)
