"""Block norms (moe_norm_*, BlockNorms) against the formulas in 64 bits, and the gradient against differences.

Tolerances. Everything is summed in fp32 and rounded once, so an output differs from the 64-bit value by half a
rounding step of its type (2^-9 relative for bf16, a few 2^-24 for fp32) plus the rounding of fp32 sums over a row
or over the tokens, bounded here by 1e-5 of the tensor's largest magnitude (thousands of terms, each off by 2^-24).
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from mixture_experts_layer_histogram_gb300 import BlockNorms
    from mixture_experts_layer_histogram_gb300 import _lib as L

EPS = 1e-6
A = 0.75


def close(got, exp, name):
    got, exp = got.double().cpu(), exp.double().cpu()
    step = 2.0 ** -8 if got_is_bf16(name[1]) else 0.0
    top = exp.abs().max().item() if exp.numel() else 0.0
    over = (got - exp).abs() - (step * exp.abs() + 1e-5 * top)
    assert torch.isfinite(got).all(), name
    assert over.numel() == 0 or over.max().item() <= 0, (name, over.max().item(), top)


def got_is_bf16(dtype):
    return dtype == torch.bfloat16


def rms(v):
    return 1 / torch.sqrt((v * v).mean(-1, keepdim=True) + EPS)


def fwd64(y, x, w_post, gate, w_next):
    out = A * x + (gate if gate is not None else 1.0) * (y * rms(y) * w_post)
    return out, (out * rms(out) * w_next if w_next is not None else None)


def make(T, d, dtype, gate, seed=0):
    g = torch.Generator().manual_seed(seed)
    def r(*s, k=1.0):
        return (torch.randn(s, generator=g) * k).to(dtype).cuda()
    return dict(x=r(T, d, k=2.0), y=r(T, d, k=0.5), w=(1 + 0.2 * r(d).float()).to(dtype), wn=(1 + 0.2 * r(d).float()).to(dtype),
                gate=None if gate is None else (r(d) if gate == "channel" else r(T, d)), dout=r(T, d), dn=r(T, d))


def d64(s):
    return {k: (None if v is None else v.double()) for k, v in s.items()}


def back64(s, out, gate, has_next):
    """The gradients by their formulas (not by autograd), from the stored out."""
    D = d64(s)
    o = out.double()
    G = D["dout"].clone()
    res = {}
    def norm_back(dn, v, w):
        r, u = rms(v), dn * w
        return r * (u - v * r * r * (u * v).mean(-1, keepdim=True)), (dn * v * r).sum(0)
    if has_next:
        g2, res["dw_next"] = norm_back(D["dn"], o, D["wn"])
        G = G + g2
    gt = D["gate"] if gate is not None else torch.ones((), dtype=torch.float64, device="cuda")
    res["dx"] = A * G
    res["dy"], res["dw_post"] = norm_back(G * gt, D["y"], D["w"])
    if gate is not None:
        dg = G * D["y"] * rms(D["y"]) * D["w"]
        res["d_gate"] = dg.sum(0) if gate == "channel" else dg
    return res


SHAPES = [(1, 1), (1, 64), (3, 31), (5, 33), (7, 257), (129, 1537), (300, 2048), (64, 4096), (2, 8192), (3, 8191), (700, 8),
          (2000, 64), (33, 5120)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,d", SHAPES)
def test_pre(T, d, dtype):
    s = make(T, d, dtype, None, seed=T + d)
    nm = BlockNorms(T, d, dtype, eps=EPS)
    x, w = s["x"].double(), s["w"].double()
    close(nm.pre(s["x"], s["w"]), x * rms(x) * w, ("n", dtype))
    for dx_in in (None, s["dout"]):
        res = nm.pre_backward(s["dn"], s["x"], s["w"], dx_in=dx_in)
        r, u = rms(x), s["dn"].double() * w
        dx = r * (u - x * r * r * (u * x).mean(-1, keepdim=True)) + (0 if dx_in is None else dx_in.double())
        close(res["dx"], dx, ("dx", dtype))
        close(res["dw"], (s["dn"].double() * x * r).sum(0), ("dw", dtype))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("gate", [None, "channel", "token"])
@pytest.mark.parametrize("has_next", [True, False])
@pytest.mark.parametrize("T,d", SHAPES)
def test_post(T, d, has_next, gate, dtype):
    s = make(T, d, dtype, gate, seed=T + d)
    nm = BlockNorms(T, d, dtype, gate=gate, res_scale=A, eps=EPS, next_norm=has_next)
    wn = s["wn"] if has_next else None
    out, n = nm.post(s["y"], s["x"], s["w"], gate=s["gate"], w_next=wn)
    D = d64(s)
    eo, en = fwd64(D["y"], D["x"], D["w"], D["gate"], D["wn"] if has_next else None)
    close(out, eo, ("out", dtype))
    assert (n is None) == (not has_next)
    if has_next:
        close(n, en, ("n", dtype))
    res = nm.post_backward(s["dout"], s["dn"] if has_next else None, out, s["y"], s["w"], gate=s["gate"], w_next=wn)
    exp = back64(s, out, gate, has_next)
    assert set(res) == set(exp)
    for k in exp:
        close(res[k], exp[k], (k, dtype))


def test_post_without_stream_gradient():
    """The top of a stack: only the next norm's output has a gradient."""
    s = make(50, 256, torch.float32, "channel")
    nm = BlockNorms(50, 256, torch.float32, gate="channel", res_scale=A, eps=EPS)
    out, _ = nm.post(s["y"], s["x"], s["w"], gate=s["gate"], w_next=s["wn"])
    res = nm.post_backward(None, s["dn"], out, s["y"], s["w"], gate=s["gate"], w_next=s["wn"])
    exp = back64(dict(s, dout=torch.zeros_like(s["dout"])), out, "channel", True)
    for k in exp:
        close(res[k], exp[k], (k, torch.float32))


def test_gradient_against_differences():
    """Directional derivatives of <dout, out> + <dn, n> by central differences in 64 bits: the step 1e-5 leaves an error
    of 1e-10 in the difference, so what is compared is the fp32 kernel's (1e-4 of the directional derivative's
    scale, the sum of the magnitudes of its terms)."""
    T, d = 17, 96
    for gate in ("channel", "token"):
        s = make(T, d, torch.float32, gate, seed=5)
        D = d64(s)
        nm = BlockNorms(T, d, torch.float32, gate=gate, res_scale=A, eps=EPS)
        out, _ = nm.post(s["y"], s["x"], s["w"], gate=s["gate"], w_next=s["wn"])
        res = nm.post_backward(s["dout"], s["dn"], out, s["y"], s["w"], gate=s["gate"], w_next=s["wn"])
        g = torch.Generator().manual_seed(1)
        for name, grad in (("x", "dx"), ("y", "dy"), ("w", "dw_post"), ("gate", "d_gate"), ("wn", "dw_next")):
            v = torch.randn(D[name].shape, generator=g, dtype=torch.float64).cuda()
            def f(h):
                P = dict(D)
                P[name] = D[name] + h * v
                o, n = fwd64(P["y"], P["x"], P["w"], P["gate"], P["wn"])
                return ((o * D["dout"]).sum() + (n * D["dn"]).sum()).item()
            num = (f(1e-5) - f(-1e-5)) / 2e-5
            got = (res[grad].double() * v)
            assert abs(got.sum().item() - num) <= 1e-4 * got.abs().sum().item(), (gate, name)


def test_rows_of_zeros_and_huge_values():
    """rms of a zero row is 1 / sqrt(eps): finite, outputs zero. Values near the top of bf16's range overflow the sum
    of squares in fp32 as in the formula: rms 0."""
    x = torch.zeros(4, 512, device="cuda")
    x[1] = 1e-30
    nm = BlockNorms(4, 512, torch.float32, eps=EPS)
    w = torch.ones(512, device="cuda")
    n = nm.pre(x, w)
    assert (n[0] == 0).all() and torch.isfinite(n).all()
    res = nm.pre_backward(torch.ones_like(x), x, w)
    assert torch.isfinite(res["dx"]).all() and abs(res["dx"][0, 0].item() - 1000.0) < 1e-2


def test_non_finite_rows_stay_in_their_row():
    s = make(6, 2048, torch.bfloat16, "channel")
    s["y"][2, 7] = float("nan")
    s["x"][4, 9] = float("inf")
    nm = BlockNorms(6, 2048, torch.bfloat16, gate="channel", res_scale=A, eps=EPS)
    out, n = nm.post(s["y"], s["x"], s["w"], gate=s["gate"], w_next=s["wn"])
    rows = torch.isfinite(n.float()).all(1).cpu().tolist()
    assert rows == [True, True, False, True, False, True]
    assert torch.isfinite(out[4].float()).sum().item() == 2047


def test_pre_output_outlives_post():
    """A block's backward may read its input again (a router's weight gradient does): post writes the next block's input
    elsewhere."""
    s = make(20, 256, torch.bfloat16, None)
    nm = BlockNorms(20, 256, torch.bfloat16, res_scale=A, eps=EPS)
    n0 = nm.pre(s["x"], s["w"])
    keep = n0.clone()
    _, n1 = nm.post(s["y"], s["x"], s["w"], w_next=s["wn"])
    assert torch.equal(n0, keep) and n1.data_ptr() != n0.data_ptr()


def test_no_tokens():
    d = 128
    nm = BlockNorms(0, d, torch.bfloat16, gate="channel", eps=EPS)
    e = torch.empty((0, d), dtype=torch.bfloat16, device="cuda")
    w = torch.ones(d, dtype=torch.bfloat16, device="cuda")
    nm.pre(e, w)
    nm.post(e, e, w, gate=w, w_next=w)
    res = nm.post_backward(e, e, e, e, w, gate=w, w_next=w)
    for k in ("dw_post", "d_gate", "dw_next"):
        assert (res[k] == 0).all()
    assert (nm.pre_backward(e, e, w)["dw"] == 0).all()


def test_same_inputs_same_bits_and_other_stream():
    s = make(3000, 2048, torch.bfloat16, "channel")
    outs = []
    side = torch.cuda.Stream()
    for stream in (None, side):
        nm = BlockNorms(3000, 2048, torch.bfloat16, gate="channel", res_scale=A, eps=EPS)
        torch.cuda.synchronize()
        out, n = nm.post(s["y"], s["x"], s["w"], gate=s["gate"], w_next=s["wn"], stream=stream)
        res = nm.post_backward(s["dout"], s["dn"], out, s["y"], s["w"], gate=s["gate"], w_next=s["wn"], stream=stream)
        torch.cuda.synchronize()
        outs.append([out.clone(), n.clone()] + [res[k].clone() for k in sorted(res)])
    for a, b in zip(*outs):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))


def test_refusals():
    d = 64
    x = torch.randn(4, d, device="cuda")
    w = torch.ones(d, device="cuda")
    n = torch.empty_like(x)
    with pytest.raises(ValueError):
        L.moe_norm_fwd(x.t().contiguous().t(), w, n)          # strides
    with pytest.raises(ValueError):
        L.moe_norm_fwd(x, w.bfloat16(), n)
    with pytest.raises(ValueError):
        L.moe_norm_fwd(x, w[:-1], n)
    with pytest.raises(TypeError):
        L.moe_norm_fwd(x.half(), w.half(), n.half())
    with pytest.raises(L.MoeError):
        L.moe_norm_fwd(x, w, n, eps=0.0)
    big = torch.randn(1, 8193, device="cuda")
    with pytest.raises(L.MoeError) as e:
        L.moe_norm_fwd(big, big[0].clone(), torch.empty_like(big))
    assert e.value.code == -2
    flat = torch.randn(4 * d + 1, device="cuda")
    with pytest.raises(L.MoeError) as e:                      # rows of 16-byte vectors on a 4-byte boundary
        L.moe_norm_fwd(flat[1:].view(4, d), w, n)
    assert e.value.code == -1
    with pytest.raises(ValueError):
        BlockNorms(4, d, gate="row")
    nm = BlockNorms(4, d, torch.float32, gate="channel")
    with pytest.raises(ValueError):
        nm.post(x, x, w, w_next=w)                            # the gate it was built for is missing
    with pytest.raises(ValueError):
        nm.post(x, x, w, gate=w)                              # the next norm's weights are missing
    with pytest.raises(RuntimeError):
        BlockNorms(4, d, torch.float32, backward=False).pre_backward(x, x, w)
