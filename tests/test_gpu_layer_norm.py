"""Layer norm (moe_layer_norm_*, LayerNorm) against its formulas in 64 bits, and the gradient against differences.

Tolerances. Statistics and sums are fp32 and every output is rounded once: an output differs from the 64-bit value by half a
rounding step of its type (bf16 has 8 significant bits: neighbours just above a power of two are 2^-7 of it apart, so half a step is
up to 2^-8 of the value; fp32 24 bits: 2^-24) and by fp32 sums over a row or over the tokens. A sum of n
terms in any order of additions is off by at most n 2^-24 of the sum of magnitudes, in practice by about sqrt(n) 2^-24 of it:
at the 8192 values or 3000 tokens here, 1e-5 of the tensor's largest magnitude covers that. The mean's error moves
z by (spread of fp32 sums) / std and is taken off again by the kernel, so offsets of the row add nothing.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from mixture_experts_layer_histogram_gb300 import LayerNorm, act8_dequantize
    from mixture_experts_layer_histogram_gb300 import _lib as L

EPS = 1e-5
SHAPES = [(1, 1), (3, 2), (1, 64), (3, 31), (4, 32), (5, 33), (7, 257), (129, 1537), (300, 2048), (64, 4096), (2, 8192), (3, 8191),
          (700, 8), (3000, 64), (33, 5120), (9, 40)]
TYPES = [torch.float32, torch.bfloat16]


def close(got, exp, name, more=0.0):
    assert got.shape == exp.shape, name
    got, exp = got.double(), exp.double()
    half = torch.finfo(name[1]).eps / 2
    top = exp.abs().max().item() if exp.numel() else 0.0
    over = (got - exp).abs() - (half * exp.abs() + (1e-5 + more) * top)
    assert torch.isfinite(got).all(), name
    assert over.numel() == 0 or over.max().item() <= 0, (name, over.max().item(), top)


def make(T, d, dtype, seed=0, offset=0.5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s, k=1.0, o=0.0: (torch.randn(s, generator=g, device="cuda") * k + o).to(dtype)  # noqa: E731
    return dict(x=r(T, d, k=2.0, o=offset), w=r(d, k=0.2, o=1.0), b=r(d, k=0.3), dn=r(T, d), dres=r(T, d))


def stats(x):
    x = x.double()
    m = x.mean(1, keepdim=True)
    return m, 1 / ((x - m).square().mean(1, keepdim=True) + EPS).sqrt()


def grads(dn, z, r, w, dres=None):
    dn, w = dn.double(), w.double()
    u = dn * w
    dx = r * (u - u.mean(1, keepdim=True) - z * (u * z).mean(1, keepdim=True))
    return dx if dres is None else dx + dres.double(), (dn * z).sum(0), dn.sum(0)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,d", SHAPES)
def test_forward_and_backward(T, d, dtype):
    s = make(T, d, dtype, T + d)
    m, r = stats(s["x"])
    z = (s["x"].double() - m) * r
    for bias in (True, False):
        nm = LayerNorm(T, d, dtype, eps=EPS, bias=bias)
        n = nm.forward(s["x"], s["w"], s["b"] if bias else None)
        close(n, z * s["w"].double() + (s["b"].double() if bias else 0), ("n", dtype))
        close(nm.mean, m[:, 0], ("mean", torch.float32))
        close(nm.rstd, r[:, 0], ("rstd", torch.float32))
        for dres in (None, s["dres"]):
            res = nm.backward(s["dn"], s["w"], x=s["x"], dx_in=dres)
            dx, dw, db = grads(s["dn"], z, r, s["w"], dres)
            close(res["dx"], dx, ("dx", dtype))
            close(res["dw"], dw, ("dw", dtype))
            assert ("db" in res) == bias
            if bias:
                close(res["db"], db, ("db", dtype))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,d", SHAPES + [(700, 33), (2435, 1023), (2435, 1537), (1300, 4089), (1300, 63), (1221, 8177), (611, 8191), (1300, 2046), (700, 1),
                                          (2000, 5), (3001, 31), (640, 3), (80001, 5), (500000, 1), (50001, 31), (150, 4001)])
def test_kept(T, d, dtype):
    s = make(T, d, dtype, T + d)
    m, r = stats(s["x"])
    z = (s["x"].double() - m) * r
    nm, plain = LayerNorm(T, d, dtype, eps=EPS, keep="f8"), LayerNorm(T, d, dtype, eps=EPS)
    n, other = nm.forward(s["x"], s["w"], s["b"]), plain.forward(s["x"], s["w"], s["b"])
    close(n, z * s["w"].double() + s["b"].double(), ("n", dtype))
    # the same kernel where rows are whole words (else the sums' order may differ: each is within the bound of the formula)
    assert torch.equal(n, other) or d * s["x"].element_size() % 16
    zq = act8_dequantize(nm.codes, nm.scales, torch.float32).double()
    # half a step of the codes (2^-4 of the value, 2^-10 of a scale that is at most max / 224), and z's own rounding
    top = torch.nn.functional.pad(z.abs(), (0, -d % 32)).view(T, -1, 32).amax(2).repeat_interleave(32, 1)[:, :d]
    assert ((zq - z).abs() <= 2.0 ** -4 * z.abs() + 2.0 ** -10 / 224 * top + 1e-5 * z.abs().max()).all()
    again = nm.restore(s["w"], s["b"], out=torch.empty_like(s["x"]))
    close(again, zq * s["w"].double() + s["b"].double(), ("again", dtype))
    assert torch.equal(nm.restore(s["w"], s["b"]), again) and nm.restore(s["w"], s["b"]) is nm.n
    for dres in (None, s["dres"]):
        res = nm.backward(s["dn"], s["w"], dx_in=dres)
        dx, dw, db = grads(s["dn"], zq, nm.rstd.double()[:, None], s["w"], dres)
        close(res["dx"], dx, ("dx", dtype))
        close(res["dw"], dw, ("dw", dtype))
        close(res["db"], db, ("db", dtype))


@pytest.mark.parametrize("d", [5, 100, 2048, 1001])
def test_rows_far_from_zero(d):
    """A mean of 3000 deviations: fp32 holds x there to 2^-12 of a deviation, and the gradients are those of what it holds."""
    s = make(33, d, torch.float32, d, offset=6000.0)
    m, r = stats(s["x"])
    z = (s["x"].double() - m) * r
    nm = LayerNorm(33, d, torch.float32, eps=EPS)
    close(nm.forward(s["x"], s["w"], s["b"]), z * s["w"].double() + s["b"].double(), ("n", torch.float32))
    res = nm.backward(s["dn"], s["w"], x=s["x"])
    dx, dw, _ = grads(s["dn"], z, r, s["w"])
    close(res["dx"], dx, ("dx", torch.float32))
    close(res["dw"], dw, ("dw", torch.float32))


def test_gradient_against_differences():
    T, d = 4, 96
    s = make(T, d, torch.float32, 3)
    nm = LayerNorm(T, d, torch.float32, eps=EPS)
    nm.forward(s["x"], s["w"], s["b"])
    res = {k: v.double() for k, v in nm.backward(s["dn"], s["w"], x=s["x"]).items()}

    def f(x, w, b):
        m, r = stats(x)
        return (s["dn"].double() * ((x - m) * r * w + b)).sum()

    v = {k: s[k].double() for k in ("x", "w", "b")}
    g = torch.Generator(device="cuda").manual_seed(8)
    for k, grad in (("x", "dx"), ("w", "dw"), ("b", "db")):
        u = torch.randn(v[k].shape, generator=g, device="cuda", dtype=torch.float64)
        h = 1e-5                                     # error of the difference: h^2, and 2^-52 of f over h
        diff = (f(**{**v, k: v[k] + h * u}) - f(**{**v, k: v[k] - h * u})) / (2 * h)
        assert abs((res[grad] * u).sum().item() - diff.item()) <= 1e-5 * (res[grad] * u).abs().sum().item()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d", [257, 2048])
def test_rows_that_overflow_and_rows_that_are_not_finite(d, dtype):
    """Squares past fp32's range count as an infinite variance; a NaN or an infinity stays in its row (and the weights' sums)."""
    T = 6
    s = make(T, d, dtype, d)
    rest = [0, 2, 4, 5]
    x = s["x"].clone()
    x[1] = x[1] * 1e25
    x[3, d // 2] = float("nan")
    for keep in (None, "f8"):
        nm, ref = LayerNorm(T, d, dtype, eps=EPS, keep=keep), LayerNorm(4, d, dtype, eps=EPS, keep=keep)
        n, want = nm.forward(x, s["w"], s["b"]), ref.forward(s["x"][rest], s["w"], s["b"])
        assert torch.equal(n[rest], want) and torch.equal(n[1], s["b"]) and n[3].isnan().all()
        a = nm.backward(s["dn"], s["w"], x=None if keep else x, dx_in=s["dres"])
        b = ref.backward(s["dn"][rest].contiguous(), s["w"], x=None if keep else s["x"][rest], dx_in=s["dres"][rest].contiguous())
        assert torch.equal(a["dx"][rest], b["dx"]) and torch.equal(a["dx"][1], s["dres"][1]) and a["dx"][3].isnan().all()
        assert a["dw"].isnan().any() and torch.isfinite(a["db"]).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d", [33, 34, 61, 63, 1023, 1537, 2045, 4082, 4089, 4095, 8177, 8186, 8191])
@pytest.mark.parametrize("T", [1, 9, 700, 2435])
def test_rows_that_start_anywhere(T, d, dtype):
    """Odd row lengths, one row per block and many, next to rows that are not finite: nothing of a neighbour's row is read into a row's
    sums, and nothing is written outside the rows."""
    s = make(T, d, dtype, T * d)
    m, r = stats(s["x"])
    z = (s["x"].double() - m) * r
    nm = LayerNorm(T, d, dtype, eps=EPS)
    room = torch.full((T * d + 64,), 7.0, dtype=dtype, device="cuda")
    nm.n = room[32:32 + T * d].view(T, d)
    nm._out[0] = nm.n.data_ptr()
    n = nm.forward(s["x"], s["w"], s["b"])
    close(n, z * s["w"].double() + s["b"].double(), ("n", dtype))
    assert room[:32].eq(7).all() and room[32 + T * d:].eq(7).all()
    res = nm.backward(s["dn"], s["w"], x=s["x"], dx_in=s["dres"])
    dx, dw, db = grads(s["dn"], z, r, s["w"], s["dres"])
    close(res["dx"], dx, ("dx", dtype))
    close(res["dw"], dw, ("dw", dtype))
    close(res["db"], db, ("db", dtype))
    if T > 8:
        want, dx = n.clone(), res["dx"].clone()
        x, bad = s["x"].clone(), torch.arange(3, T, 5, device="cuda")
        x[bad] = float("inf")
        ok = torch.ones(T, dtype=torch.bool, device="cuda")
        ok[bad] = False
        n, res = nm.forward(x, s["w"], s["b"]), nm.backward(s["dn"], s["w"], x=x, dx_in=s["dres"])
        assert torch.equal(n[ok], want[ok]) and n[bad].isnan().all() and torch.equal(res["dx"][ok], dx[ok])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,d", [(2431, 1024), (1300, 2048), (611, 4096), (1223, 1537), (1300, 2045), (2431, 97)])
def test_many_rows_some_not_finite(T, d, dtype):
    """Rows that share a block's reductions: what stands in one changes no bit of the others, whatever their number."""
    s = make(T, d, dtype, T)
    x, bad = s["x"].clone(), torch.arange(5, T, 7, device="cuda")
    x[bad] = float("nan")
    ok = torch.ones(T, dtype=torch.bool, device="cuda")
    ok[bad] = False
    m, r = stats(s["x"])
    for keep in (None, "f8"):
        nm, ref = LayerNorm(T, d, dtype, eps=EPS, keep=keep), LayerNorm(T, d, dtype, eps=EPS, keep=keep)
        n, want = nm.forward(x, s["w"], s["b"]), ref.forward(s["x"], s["w"], s["b"])
        close(want, (s["x"].double() - m) * r * s["w"].double() + s["b"].double(), ("n", dtype))
        assert torch.equal(n[ok], want[ok]) and n[bad].isnan().all() and torch.equal(nm.rstd[ok], ref.rstd[ok])
        if keep:
            assert torch.equal(nm.codes[ok], ref.codes[ok]) and nm.codes[bad].eq(0).all()


@pytest.mark.parametrize("dtype", TYPES)
def test_no_tokens(dtype):
    for keep in (None, "f8"):
        nm = LayerNorm(0, 96, dtype, keep=keep)
        e, w = torch.empty(0, 96, dtype=dtype, device="cuda"), torch.ones(96, dtype=dtype, device="cuda")
        nm.dw.fill_(7)
        nm.db.fill_(7)
        assert nm.forward(e, w, w).shape == (0, 96)
        res = nm.backward(e, w, x=None if keep else e)
        assert res["dw"].eq(0).all() and res["db"].eq(0).all()


@pytest.mark.parametrize("keep", [None, "f8"])
@pytest.mark.parametrize("d", [1000, 1001])
def test_in_place_repeatable_and_rows_behind(d, keep):
    """dx over dx_in, the same bits twice, and nothing written past the last row."""
    T = 200
    s = make(T, d, torch.bfloat16, 1)
    nm = LayerNorm(T, d, eps=EPS, keep=keep)
    nm.forward(s["x"], s["w"], s["b"])
    x = None if keep else s["x"]
    first = {k: v.clone() for k, v in nm.backward(s["dn"], s["w"], x=x, dx_in=s["dres"]).items()}
    room = torch.full((T + 8, d), 9.0, dtype=torch.bfloat16, device="cuda")
    room[:T] = s["dres"]
    L.moe_layer_norm_bwd(s["dn"], x, nm.codes, nm.scales, nm.mean, nm.rstd, s["w"], room[:T], room[:T], nm.dw, nm.db, nm.ws, EPS)
    assert torch.equal(room[:T], first["dx"]) and room[T:].eq(9).all()
    assert torch.equal(nm.dw, first["dw"]) and torch.equal(nm.db, first["db"])
    n = torch.full((T + 8, d), 9.0, dtype=torch.bfloat16, device="cuda")
    L.moe_layer_norm_fwd(s["x"], s["w"], s["b"], n[:T], eps=EPS)
    assert torch.equal(n[:T], nm.n) and n[T:].eq(9).all()


@pytest.mark.parametrize("keep", [None, "f8"])
def test_stream_and_graph(keep):
    T, d = 77, 512
    s = make(T, d, torch.bfloat16, 5)
    nm, ref = (LayerNorm(T, d, eps=EPS, keep=keep) for _ in range(2))

    def step(nm, x, stream=None):
        n = nm.forward(x, s["w"], s["b"], stream=stream)
        return [n] + list(nm.backward(s["dn"], s["w"], x=None if keep else x, dx_in=s["dres"], stream=stream).values())

    want = [t.clone() for t in step(ref, s["x"])]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = step(nm, s["x"], side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    x = s["x"].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(nm, x)
    x.copy_(s["dn"])
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(got, step(ref, s["dn"])))
