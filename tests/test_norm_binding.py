"""BlockNorms.post and moe_norm_residual_fwd make the C call in one place, with one set of checks. (No GPU needed: the
tensors only claim to be on one, and the call is recorded.)"""
import pytest
import torch

from mixture_experts_layer_histogram_gb300 import BlockNorms
from mixture_experts_layer_histogram_gb300 import _lib as L

T, D = 3, 64


class Claimed:
    def __init__(self, *shape, dtype=torch.float32):
        self._t, self.is_cuda = torch.zeros(shape, dtype=dtype), True

    def __getattr__(self, name):
        return getattr(self._t, name)


@pytest.fixture
def calls(monkeypatch):
    seen = []

    class Lib:
        def moe_norm_residual_fwd(self, *args):
            seen.append(args)
            return 0

    monkeypatch.setattr(L, "lib", Lib)
    monkeypatch.setattr(L, "_s", lambda stream: 0)
    real, through = L.norm_residual_fwd_into, []
    monkeypatch.setattr(L, "norm_residual_fwd_into", lambda *a, **k: (through.append(1), real(*a, **k)))
    yield seen
    assert len(through) >= len(seen)


def norms(gate, next_norm):
    nm = BlockNorms.__new__(BlockNorms)
    nm.T, nm.d, nm.dtype, nm.gate_kind, nm.next_norm, nm.res_scale, nm.eps = T, D, torch.float32, gate, next_norm, 0.5, 1e-6
    nm.out, nm.n = Claimed(T, D), Claimed(T, D) if next_norm else None
    nm._kind = {None: 0, "channel": 1, "token": 2}[gate]
    nm._out_ptr, nm._n_ptr = nm.out.data_ptr(), nm.n.data_ptr() if next_norm else None
    return nm


@pytest.mark.parametrize("next_norm", [True, False])
@pytest.mark.parametrize("gate,shape,kind", [(None, None, 0), ("channel", (D,), 1), ("token", (T, D), 2)])
def test_one_binding(calls, gate, shape, kind, next_norm):
    nm, y, x, w = norms(gate, next_norm), Claimed(T, D), Claimed(T, D), Claimed(D)
    g, wn = Claimed(*shape) if gate else None, Claimed(D) if next_norm else None
    out, n = nm.post(y, x, w, gate=g, w_next=wn)
    assert out is nm.out and n is nm.n
    p = lambda t: None if t is None else t.data_ptr()   # noqa: E731
    want = (p(y), p(x), p(w), p(g), kind, p(wn), T, D, 0, 0.5, 1e-6, p(out), p(n), 0)
    L.moe_norm_residual_fwd(y, x, w, g, wn, nm.out, nm.n, 0.5, 1e-6)
    assert calls == [want, want]


def test_refusals(calls):
    nm, y, x, w = norms("channel", True), Claimed(T, D), Claimed(T, D), Claimed(D)
    ok = dict(gate=w, w_next=w)
    for args, kw in (((Claimed(T, D - 1), x, w), ok), ((y, Claimed(T + 1, D), w), ok), ((y, x, Claimed(D + 1)), ok),
                     ((y, x, Claimed(D, dtype=torch.bfloat16)), ok), ((y, x, w), dict(gate=None, w_next=w)),
                     ((y, x, w), dict(gate=Claimed(T, D), w_next=w)), ((y, x, w), dict(gate=w)),
                     ((y, x, w), dict(gate=Claimed(D + 1), w_next=w)), ((y, x, w), dict(gate=w, w_next=Claimed(2 * D))),
                     (tuple(Claimed(*t.shape, dtype=torch.bfloat16) for t in (y, x, w)), ok),
                     ((torch.zeros(T, D), x, w), ok)):
        with pytest.raises(ValueError):
            nm.post(*args, **kw)
    for out, n in ((Claimed(T, D + 1), Claimed(T, D)), (Claimed(T, D), Claimed(T, D, dtype=torch.bfloat16)), (Claimed(T, D), None)):
        with pytest.raises(ValueError):
            L.moe_norm_residual_fwd(y, x, w, w, w, out, n)
    assert calls == []
