"""Arguments that the layer norm and the 8-bit activations refuse on the host (no GPU needed)."""
import ctypes
import os

import pytest
import torch

FAKE = ctypes.c_void_p(1 << 20)   # never dereferenced: every call below fails validation first
ODD = ctypes.c_void_p((1 << 20) + 4)
NULL = None


@pytest.fixture(scope="module")
def L():
    from mixture_experts_layer_histogram_gb300 import _lib, build
    if not os.path.exists(_lib.LIB_PATH):
        build.build()
    return _lib.lib()


def test_act8_refusals(L):
    assert [L.moe_act8_scale_bytes(r, k) for r, k in ((0, 5), (3, 1), (3, 32), (3, 33), (-1, 4), (4, 0))] == [0, 3, 3, 6, 0, 0]
    for q in (lambda *a, x=FAKE, c=FAKE, s=FAKE: L.moe_act8_quantize(x, a[0], a[1], a[2], c, s, NULL),
              lambda *a, x=FAKE, c=FAKE, s=FAKE: L.moe_act8_dequantize(c, s, a[1], a[2], a[0], x, NULL)):
        assert q(2, 4, 64) == -1 and q(0, -1, 64) == -1 and q(0, 4, 0) == -1
        assert q(0, 1 << 40, 64) == -2
        for bad in (NULL, ODD):
            assert q(0, 4, 64, x=bad) == -1 and q(0, 4, 64, c=bad) == -1 and q(0, 4, 64, s=bad) == -1
        assert q(0, 0, 64, x=NULL, c=NULL, s=NULL) == 0


def test_layer_norm_refusals(L):
    def fwd(x=FAKE, w=FAKE, b=FAKE, T=4, d=64, dtype=0, eps=1e-5, n=FAKE, mean=FAKE, rstd=FAKE, codes=NULL, scales=NULL):
        return L.moe_layer_norm_fwd(x, w, b, T, d, dtype, eps, n, mean, rstd, codes, scales, NULL)
    assert fwd(d=0) == fwd(T=-1) == fwd(dtype=2) == fwd(eps=0.0) == fwd(eps=float("nan")) == -1
    assert fwd(d=8193) == -2
    for k in ("x", "w", "n"):
        assert fwd(**{k: NULL}) == fwd(**{k: ODD}) == -1
    for k in ("b", "mean", "rstd"):
        assert fwd(**{k: ODD}) == -1
    assert fwd(codes=FAKE) == fwd(scales=FAKE) == fwd(codes=ODD, scales=FAKE) == -1
    assert fwd(T=0, x=NULL, w=NULL, n=NULL) == 0

    def restore(codes=FAKE, scales=FAKE, w=FAKE, b=NULL, T=4, d=64, dtype=0, n=FAKE):
        return L.moe_layer_norm_restore(codes, scales, w, b, T, d, dtype, n, NULL)
    for k in ("codes", "scales", "w", "n"):
        assert restore(**{k: NULL}) == restore(**{k: ODD}) == -1
    assert restore(b=ODD) == restore(d=0) == restore(dtype=3) == -1 and restore(d=9000) == -2 and restore(T=0) == 0

    ws = L.moe_layer_norm_bwd_workspace_size(4, 64, 0)
    assert ws >= 2 * 4 * 64 * 4 and L.moe_layer_norm_bwd_workspace_size(0, 64, 0) >= 2 * 64 * 4
    assert L.moe_layer_norm_bwd_workspace_size(4, 8193, 0) == L.moe_layer_norm_bwd_workspace_size(4, 64, 5) == 0

    def bwd(dn=FAKE, x=FAKE, codes=NULL, scales=NULL, mean=FAKE, rstd=FAKE, w=FAKE, dx_in=NULL, T=4, d=64, dtype=0, eps=1e-5,
            dx=FAKE, dw=FAKE, db=FAKE, wsp=FAKE, n=ws):
        return L.moe_layer_norm_bwd(dn, x, codes, scales, mean, rstd, w, dx_in, T, d, dtype, eps, dx, dw, db, wsp, n, NULL)
    for k in ("dn", "x", "mean", "rstd", "w", "dx", "dw", "wsp"):
        assert bwd(**{k: NULL}) == bwd(**{k: ODD}) == -1, k
    assert bwd(dx_in=ODD) == bwd(db=ODD) == bwd(n=ws - 1) == bwd(wsp=ctypes.c_void_p((1 << 20) + 16)) == -1
    assert bwd(codes=FAKE) == bwd(scales=FAKE) == bwd(codes=FAKE, scales=FAKE) == -1     # x as well as codes; one of the two
    assert bwd(x=NULL, codes=FAKE, scales=ODD) == -1
    assert bwd(T=-1) == bwd(dtype=2) == bwd(eps=0.0) == -1 and bwd(d=8193) == -2


class Claimed:
    """A CPU tensor that says it is on a CUDA device."""

    def __init__(self, *shape, dtype=torch.float32, device=0):
        self._t, self.is_cuda, self._dev = torch.zeros(shape, dtype=dtype), True, device

    def get_device(self):
        return self._dev

    def __getattr__(self, name):
        return getattr(self._t, name)


@pytest.fixture
def B(monkeypatch):
    """The binding, with tensors that only claim to be on a GPU and a library that records calls."""
    from mixture_experts_layer_histogram_gb300 import _lib as B

    class Lib:
        calls = []

        def __getattr__(self, name):
            return lambda *a: (self.calls.append((name, a)), 0)[1]

    monkeypatch.setattr(B, "lib", Lib)
    monkeypatch.setattr(B, "_s", lambda stream: 0)
    monkeypatch.setattr(B, "_device", lambda: 0)
    Lib.calls.clear()
    B_calls = Lib.calls
    yield B, B_calls


def test_binding_refusals(B):
    B, calls = B
    u8 = torch.uint8
    good = dict(x=Claimed(4, 64), codes=Claimed(4, 64, dtype=u8), scales=Claimed(8, dtype=u8))
    B.moe_act8_quantize(**good)
    B.moe_act8_dequantize(good["codes"], good["scales"], good["x"])
    norm = dict(x=Claimed(4, 64), w=Claimed(64), b=Claimed(64), n=Claimed(4, 64), mean=Claimed(4), rstd=Claimed(4),
                codes=Claimed(4, 64, dtype=u8), scales=Claimed(8, dtype=u8))
    B.moe_layer_norm_fwd(**norm)
    back = dict(dn=Claimed(4, 64), x=Claimed(4, 64), codes=None, scales=None, mean=Claimed(4), rstd=Claimed(4), w=Claimed(64),
                dx_in=Claimed(4, 64), dx=Claimed(4, 64), dw=Claimed(64), db=Claimed(64), ws=Claimed(64, dtype=u8))
    B.moe_layer_norm_bwd(**back)
    rest = dict(codes=norm["codes"], scales=norm["scales"], w=Claimed(64), b=None, n=Claimed(4, 64))
    B.moe_layer_norm_restore(**rest)
    n = len(calls)
    assert n == 5
    for fn, args in ((B.moe_act8_quantize, good), (B.moe_layer_norm_fwd, norm), (B.moe_layer_norm_bwd, back),
                     (B.moe_layer_norm_restore, rest)):
        for k, t in args.items():
            if t is None or k in ("x", "dn", "ws") and fn is not B.moe_layer_norm_bwd:
                continue
            shape = tuple(t.shape)
            wrong = [Claimed(*shape, dtype=t.dtype, device=1)]
            if k != "ws":
                wrong += [Claimed(*shape, dtype=torch.float64), Claimed(*(s - 1 for s in shape), dtype=t.dtype)]
                if len(shape) == 2:
                    strided = Claimed(shape[0], 2 * shape[1], dtype=t.dtype)
                    strided._t = strided._t[:, ::2]
                    wrong.append(strided)
            for bad in wrong:
                with pytest.raises((ValueError, TypeError)):
                    fn(**{**args, k: bad})
    assert len(calls) == n


def test_class_refusals():
    from mixture_experts_layer_histogram_gb300 import LayerNorm
    with pytest.raises(ValueError, match="keep"):
        LayerNorm(4, 64, keep="f4")
    with pytest.raises(ValueError, match="backward"):
        LayerNorm(4, 64, keep="f8", backward=False)
    nm = LayerNorm.__new__(LayerNorm)
    nm.bias, nm.keep, nm.backward_enabled = True, "f8", True
    with pytest.raises(ValueError, match="bias"):
        nm.forward(None, None)
    with pytest.raises(ValueError, match="x is needed"):
        nm.backward(None, None, x=1)
    nm.keep = None
    with pytest.raises(ValueError, match="x is needed"):
        nm.backward(None, None)
    with pytest.raises(RuntimeError, match="nothing"):
        nm.restore(None)
    nm.backward_enabled = False
    with pytest.raises(RuntimeError, match="backward"):
        nm.backward(None, None)
