"""Two sets of buffers in turn on one object: what each micro-batch keeps is what its backward reads."""
import copy

import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from mixture_experts_layer_histogram_gb300 import GatedFFN, LayerNorm

BF = torch.bfloat16


def randn(seed, *shapes):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [torch.randn(s, generator=g, device="cuda").to(BF) for s in shapes]


@pytest.mark.parametrize("keep", [None, "f8"])
def test_layer_norm(keep):
    T, d = 100, 320
    w, b = randn(0, d, d)
    nm, refs = LayerNorm(T, d, keep=keep), [LayerNorm(T, d, keep=keep) for _ in range(2)]
    data, kept = [randn(i + 1, (T, d), (T, d)) for i in range(2)], []
    names = ("n", "rstd") + (("codes", "scales") if keep else ("mean",))
    for (x, _), ref in zip(data, refs):
        own = {k: torch.empty_like(getattr(nm, k)) for k in names}
        for k, t in own.items():
            setattr(nm, k, t)
        assert nm.forward(x, w, b) is own["n"] and torch.equal(own["n"], ref.forward(x, w, b))
        kept.append(own)
    for (x, dn), ref, own in list(zip(data, refs, kept)):
        for k, t in own.items():
            setattr(nm, k, t)
        nm.dx = torch.empty_like(nm.dx)
        got, want = nm.backward(dn, w, x=None if keep else x), ref.backward(dn, w, x=None if keep else x)
        assert got["dx"] is nm.dx and all(torch.equal(got[k], want[k]) for k in want)
        if keep:
            assert torch.equal(nm.restore(w, b), ref.restore(w, b))


@pytest.mark.parametrize("keep", [None, "f8"])
def test_gated_ffn(keep):
    T, d, f = 150, 128, 96
    wgu, wd = randn(0, (2 * f, d), (d, f))
    ffn, refs = GatedFFN(T, d, f, keep=keep), [GatedFFN(T, d, f, keep=keep) for _ in range(2)]
    data, kept = [randn(i + 1, (T, d), (T, d)) for i in range(2)], []
    names = ("ab", "ab_scales") if keep else ("ab", "h")
    for (x, _), ref in zip(data, refs):
        own = {k: torch.empty_like(getattr(ffn, k)) for k in names + ("y",)}
        for k, t in own.items():
            setattr(ffn, k, t)
        assert ffn.forward(x, wgu, wd) is own["y"] and torch.equal(own["y"], ref.forward(x, wgu, wd))
        kept.append(own)
    for (x, dy), ref, own in zip(data, refs, kept):
        for k in names:
            setattr(ffn, k, own[k])
        for k in ("dab", "dx", "dw_gate_up", "dw_down"):
            setattr(ffn, k, torch.empty_like(getattr(ffn, k)))
        ffn.ws = torch.zeros_like(ffn.ws)
        got, want = ffn.backward(dy, x, wgu, wd), ref.backward(dy, x, wgu, wd)
        assert all(got[k] is getattr(ffn, k) and torch.equal(got[k], want[k]) for k in want)
    for name, bad in (("ab", torch.empty(T, f, dtype=BF, device="cuda")), ("y", ffn.y.cpu()), ("h", ffn.h.T)):
        with pytest.raises(ValueError, match=name):
            setattr(ffn, name, bad)


@pytest.mark.parametrize("keep", [None, "f8"])
def test_deep_copies(keep):
    """A copy writes into buffers of its own, and leaves the original's alone."""
    T, d, f = 70, 128, 64
    w, b, wgu, wd, x, z, dy = randn(0, d, d, (2 * f, d), (d, f), (T, d), (T, d), (T, d))
    nm, ffn = LayerNorm(T, d, keep=keep), GatedFFN(T, d, f, keep=keep)

    def step(norm, block, x):
        n = norm.forward(x, w, b)
        y = block.forward(n, wgu, wd)
        g = block.backward(dy, n, wgu, wd)
        return [n, y, *g.values(), *norm.backward(g["dx"], w, x=None if keep else x).values()]

    first = step(nm, ffn, x)
    kept = [t.clone() for t in first]
    other = [t.clone() for t in step(copy.deepcopy(nm), copy.deepcopy(ffn), z)]
    assert all(torch.equal(a, k) for a, k in zip(first, kept))
    assert all(torch.equal(a, k) for a, k in zip(step(nm, ffn, z), other))
