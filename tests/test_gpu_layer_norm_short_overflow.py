"""Rows of at most 32 values whose squared deviations pass fp32's range: the backward, which forms such rows' statistics again in 64
bits, takes them as the forward does, z = 0 and r = 0."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from mixture_experts_layer_histogram_gb300 import LayerNorm


@pytest.mark.parametrize("keep", [None, "f8"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("d", [2, 5, 8, 31, 32, 33, 40])
def test_both_directions_agree(d, dtype, keep):
    T, bad = 6, [1, 4]
    g = torch.Generator(device="cuda").manual_seed(d)
    r = lambda *s: torch.randn(s, generator=g, device="cuda").to(dtype)  # noqa: E731
    x, w, b, dn, dres = r(T, d), r(d), r(d), r(T, d), r(T, d)
    x[bad] = x[bad] * 1e25                                  # deviations of 1e24 and more: squares above 3.4e38
    assert ((x[bad].double() - x[bad].double().mean(1, keepdim=True)).abs().amax(1) > 1e21).all()
    rest = [i for i in range(T) if i not in bad]
    nm, ref = LayerNorm(T, d, dtype, keep=keep), LayerNorm(len(rest), d, dtype, keep=keep)
    n, want = nm.forward(x, w, b), ref.forward(x[rest], w, b)
    assert torch.equal(n[rest], want) and all(torch.equal(n[i], b) for i in bad) and nm.rstd[bad].eq(0).all()
    for dx_in in (None, dres):
        got = nm.backward(dn, w, x=None if keep else x, dx_in=dx_in)
        exp = ref.backward(dn[rest].contiguous(), w, x=None if keep else x[rest], dx_in=None if dx_in is None else dx_in[rest].contiguous())
        assert torch.equal(got["dx"][rest], exp["dx"])
        assert torch.equal(got["dx"][bad], torch.zeros_like(dres[bad]) if dx_in is None else dres[bad])
        assert torch.equal(got["dw"], exp["dw"])            # a row per block: the bad rows add zeros to sums taken in order
        # db takes all rows of dn: 6 fp32 additions, rounded once
        db, size = dn.double().sum(0), dn.double().abs().sum(0)
        assert ((got["db"].double() - db).abs() <= torch.finfo(dtype).eps / 2 * db.abs() + 6 * 2.0 ** -24 * size).all()
