"""The dense block's operators on tensors of more than 2^31 values: the rows around the 2^31st value and at both ends against their
formulas, and gradients that only those rows have.

Tolerances: those of test_gpu_layer_norm.py and test_gpu_ffn.py. Where dn (dy) is zero a row gives nothing to dx and to the weight
gradients, exactly, so their sums are those of the few rows that are not."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from mixture_experts_layer_histogram_gb300 import GatedFFN, LayerNorm, act8_dequantize

    from test_gpu_ffn import gate, product, within
    from test_gpu_layer_norm import close, grads, make, stats

BF, F32 = torch.bfloat16, torch.float32


def some_rows(T, width):
    """Rows at both ends, around each multiple of 2^31 values, and a few between."""
    at = {0, 1, T - 2, T - 1, *range(17, T, T // 23)}
    for k in range(1, T * width // 2 ** 31 + 1):
        at |= {k * 2 ** 31 // width + i for i in (-1, 0, 1)}
    return torch.tensor(sorted(i for i in at if 0 <= i < T), device="cuda")


@pytest.mark.parametrize("keep", [None, "f8"])
@pytest.mark.parametrize("d", [8000, 8001])
def test_layer_norm(d, keep):
    T = 300001
    assert T * d > 2 ** 31
    rows = some_rows(T, d)
    s = make(1, d, BF, d)
    x = torch.empty(T, d, dtype=BF, device="cuda").normal_(0.5, 2.0)
    dres = torch.empty(T, d, dtype=BF, device="cuda").normal_()
    dn = torch.zeros(T, d, dtype=BF, device="cuda")
    dn[rows] = torch.randn(len(rows), d, device="cuda").to(BF)
    nm = LayerNorm(T, d, keep=keep)
    n = nm.forward(x, s["w"], s["b"])
    m, r = stats(x[rows])
    z, (w, b) = (x[rows].double() - m) * r, (s["w"].double(), s["b"].double())
    close(n[rows], z * w + b, ("n", BF))
    close(nm.rstd[rows], r[:, 0], ("rstd", F32))
    if keep:
        nb = -(-d // 32)
        z = act8_dequantize(nm.codes[rows], nm.scales.view(T, nb)[rows].flatten(), F32).double()
        close(nm.restore(s["w"], s["b"])[rows], z * w + b, ("restored", BF))
    res = nm.backward(dn, s["w"], x=None if keep else x, dx_in=dres)
    dx, dw, db = grads(dn[rows], z, nm.rstd[rows].double()[:, None] if keep else r, s["w"], dres[rows])
    close(res["dx"][rows], dx, ("dx", BF))
    close(res["dw"], dw, ("dw", BF))
    close(res["db"], db, ("db", BF))
    res["dx"][rows] = dres[rows]
    assert torch.equal(res["dx"], dres)


@pytest.mark.parametrize("T,d,f,dtype,keep", [(300001, 64, 8192, BF, None), (300001, 64, 8192, BF, "f8"), (300001, 8192, 64, BF, None),
                                              (140001, 16, 16385, F32, None), (140001, 16385, 16, F32, None)])
def test_ffn(T, d, f, dtype, keep):
    assert T * max(d, f) > 2 ** 31
    rows = some_rows(T, max(d, f))
    new = lambda *s, k=1.0: torch.empty(s, dtype=dtype, device="cuda").normal_(0.0, k)  # noqa: E731
    x, wgu, wd, add = new(T, d), new(2 * f, d, k=d ** -0.5), new(d, f, k=f ** -0.5), new(T, d)
    dy = torch.zeros(T, d, dtype=dtype, device="cuda")
    dy[rows] = new(len(rows), d)
    ffn = GatedFFN(T, d, f, dtype, keep=keep)
    y = ffn.forward(x, wgu, wd, add=add)
    xr, w64 = x[rows].double(), wgu.double()
    ab = xr @ w64.T
    noise = 4 * ((d / 16 + 16) * 2.0 ** -23 if dtype == BF else (d + 16) * 2.0 ** -24) * torch.sqrt((xr * xr) @ (w64 * w64).T)
    g, dg = gate(ab[:, :f], "silu")
    b = ab[:, f:]
    within("h", ffn.h[rows], g * b, (dg.abs() * b.abs() + 1e-2) * noise[:, :f] + g.abs() * noise[:, f:] + 1e-5 * (ab[:, :f] * b).abs() + 1e-30)
    if keep:
        kept = act8_dequantize(ffn.ab[rows], ffn.ab_scales.view(T, -1)[rows].flatten(), F32).double()
        top = ab.abs().view(len(rows), -1, 32).amax(2).repeat_interleave(32, 1)
        assert ((kept - ab).abs() <= 2.0 ** -4 * ab.abs() + 2.0 ** -10 / 224 * top + 2 * noise).all()
        ab = kept
    else:
        within("ab", ffn.ab[rows], ab, noise)
        ab = ffn.ab[rows].double()
    product("y", y[rows], ffn.h[rows], wd, dtype, add[rows])
    res = ffn.backward(dy, x, wgu, wd, add=add)
    assert ffn.status() == 0
    (g, dg), b, dyr, wd64 = gate(ab[:, :f], "silu"), ab[:, f:], dy[rows].double(), wd.double()
    dh = dyr @ wd64
    noise = 4 * ((d / 16 + 16) * 2.0 ** -23 if dtype == BF else (d + 16) * 2.0 ** -24) * torch.sqrt((dyr * dyr) @ (wd64 * wd64))
    dab = ffn.dab[rows]
    within("da", dab[:, :f], dh * b * dg, (b * dg).abs() * noise + 1e-5 * (dh * b).abs() * (1 + ab[:, :f].abs()) + 1e-30)
    within("db", dab[:, f:], dh * g, g.abs() * noise + 1e-5 * (dh * ab[:, :f]).abs() + 1e-30)
    product("dx", res["dx"][rows], dab, wgu.T, dtype, add[rows])
    product("dw_gate_up", res["dw_gate_up"], dab.T, x[rows].T, dtype)
    product("dw_down", res["dw_down"], dy[rows].T, ffn.h[rows].T, dtype)
    res["dx"][rows] = add[rows]
    assert torch.equal(res["dx"], add)
    ffn.dab[rows] = 0
    assert ffn.dab.count_nonzero() == 0
