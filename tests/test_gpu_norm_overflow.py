"""Rows whose sum of squares passes fp32's range (magnitudes above about 1e19): rms is 0 there, so the norm's output and its
gradients are zeros, what passes by the norm is untouched, and other rows do not notice. Rows of at most 32 values are
differentiated in 64 bits, where nothing overflows: their gradients are the formulas'."""
import pytest
import torch

from test_gpu_norm import A, back64, close, rms

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from mixture_experts_layer_histogram_gb300 import BlockNorms

T, HOT = 6, 3
REST = [i for i in range(T) if i != HOT]


def inputs(big, d, dtype):
    g = torch.Generator(device="cuda").manual_seed(d)
    s = {k: torch.randn(T, d, generator=g, device="cuda").to(dtype) for k in ("x", "y", "dn", "dout")}
    s["w"] = (1 + torch.rand(d, generator=g, device="cuda")).to(dtype)
    huge = {k: s[k].clone() for k in ("x", "y")}
    for k in huge:
        huge[k][HOT] = s[k][HOT] * big + big
    return s, huge


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("d", [31, 257, 2048])
@pytest.mark.parametrize("big", [1e25, 1e30])
def test_forward(big, d, dtype):
    s, huge = inputs(big, d, dtype)
    x, y, w = s["x"], s["y"], s["w"]
    nm, ref = (BlockNorms(t, d, dtype, gate="channel", res_scale=A) for t in (T, T - 1))
    n = nm.pre(huge["x"], w)
    assert n[HOT].eq(0).all() and torch.equal(n[REST], ref.pre(x[REST], w))
    o2, n2 = ref.post(y[REST], x[REST], w, gate=w, w_next=w)
    out, n = nm.post(huge["y"], x, w, gate=w, w_next=w)
    assert torch.equal(out[HOT], (x[HOT].float() * A).to(dtype)) and torch.equal(out[REST], o2) and torch.equal(n[REST], n2)
    out, n = nm.post(y, huge["x"], w, gate=w, w_next=w)
    assert n[HOT].eq(0).all() and torch.isfinite(out.float()).all() and torch.equal(out[REST], o2) and torch.equal(n[REST], n2)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("d", [257, 2048])
@pytest.mark.parametrize("big", [1e25, 1e30])
def test_backward(big, d, dtype):
    s, huge = inputs(big, d, dtype)
    x, y, w, dn, dout = s["x"], s["y"], s["w"], s["dn"], s["dout"]
    nm, ref = (BlockNorms(t, d, dtype, gate="channel", res_scale=A) for t in (T, T - 1))
    a, b = nm.pre_backward(dn, huge["x"], w, dx_in=dout), ref.pre_backward(dn[REST], x[REST], w, dx_in=dout[REST])
    assert torch.equal(a["dx"][HOT], dout[HOT]) and torch.equal(a["dx"][REST], b["dx"]) and torch.equal(a["dw"], b["dw"])
    o2, _ = ref.post(y[REST], x[REST], w, gate=w, w_next=w)
    b = ref.post_backward(dout[REST], dn[REST], o2, y[REST], w, gate=w, w_next=w)
    out, _ = nm.post(huge["y"], x, w, gate=w, w_next=w)
    a = nm.post_backward(dout, dn, out, huge["y"], w, gate=w, w_next=w)
    assert a["dy"][HOT].eq(0).all() and torch.equal(a["dy"][REST], b["dy"]) and torch.equal(a["dx"][REST], b["dx"])
    assert torch.equal(a["dw_post"], b["dw_post"]) and torch.equal(a["d_gate"], b["d_gate"])
    out, _ = nm.post(y, huge["x"], w, gate=w, w_next=w)
    a = nm.post_backward(dout, dn, out, y, w, gate=w, w_next=w)
    assert torch.equal(a["dx"][HOT], (dout[HOT].float() * A).to(dtype)) and torch.equal(a["dx"][REST], b["dx"])
    assert torch.equal(a["dw_next"], b["dw_next"]) and torch.isfinite(a["dy"].float()).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("big", [1e25, 1e30])
def test_backward_of_narrow_rows(big, dtype):
    d = 31
    s, huge = inputs(big, d, dtype)
    nm = BlockNorms(T, d, dtype, gate="channel", res_scale=A)
    a = nm.pre_backward(s["dn"], huge["x"], s["w"], dx_in=s["dout"])
    x, w, dn = huge["x"].double(), s["w"].double(), s["dn"].double()
    r, u = rms(x), dn * w
    close(a["dx"], r * (u - x * r * r * (u * x).mean(-1, keepdim=True)) + s["dout"].double(), ("dx", dtype))
    close(a["dw"], (dn * x * r).sum(0), ("dw", dtype))
    for k in ("x", "y"):
        p = dict(s, gate=s["w"], wn=s["w"], **{k: huge[k]})
        out, _ = nm.post(p["y"], p["x"], s["w"], gate=s["w"], w_next=s["w"])
        a = nm.post_backward(s["dout"], s["dn"], out, p["y"], s["w"], gate=s["w"], w_next=s["w"])
        for name, exp in back64(p, out, "channel", True).items():
            close(a[name], exp, (name, dtype))
