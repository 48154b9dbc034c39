"""The gated feed-forward block (moe_ffn_*, GatedFFN), each product against 64 bits on the operands that the kernels had.

Tolerances. Every stored value is checked from the stored values before it, so roundings do not add up: a value is off by half a
step of its type (eps / 2 of it) and by the fp32 accumulation of a sum of K products. The tensor cores add 16 products at a time
to the accumulator and cut or round the result to 24 bits: each of the K / 16 steps is off by at most 2^-23 of the partial sum, and
a partial sum of products p_k of unlike signs stays below 4 sqrt(sum p_k^2) but for rare chances; 16 steps more allow for the
parts of a cut product and the addend. fp32 adds one product at a time: K steps of 2^-24. The gate: exp and the reciprocal are
good to a few 2^-23 and the argument's size (below 20) times 2^-24, so 1e-5 of the gate's terms covers it.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from mixture_experts_layer_histogram_gb300 import GatedFFN, act8_dequantize
    from mixture_experts_layer_histogram_gb300 import _lib as L

BF, F32 = torch.bfloat16, torch.float32
C = math.sqrt(2 / math.pi)
PARTS = 4 * 76 * 16 * 8     # bytes of the arrival counts of parts


def gate(a, act):
    """act(a) and act'(a) in 64 bits."""
    if act == "silu":
        s = torch.sigmoid(a)
        return a * s, s * (1 + a * (1 - s))
    t = torch.tanh(C * (a + 0.044715 * a ** 3))
    return 0.5 * a * (1 + t), 0.5 * (1 + t) + 0.5 * a * (1 - t * t) * C * (1 + 3 * 0.044715 * a * a)


def within(name, got, exp, slack):
    assert got.shape == exp.shape and torch.isfinite(got.double()).all(), name
    over = (got.double() - exp).abs() - (torch.finfo(got.dtype).eps / 2 * exp.abs() + slack)
    assert over.max().item() <= 0, (name, over.max().item(), exp.abs().max().item())


def product(name, got, A, B, dtype, add=None):
    """got = A B^T (+ add), A [M, K] and B [N, K] as the kernel had them."""
    A, B = A.double(), B.double()
    exp, K = A @ B.T, A.shape[1]
    step = (K / 16 + 16) * 2.0 ** -23 if dtype == BF else (K + 16) * 2.0 ** -24
    size = torch.sqrt((A * A) @ (B * B).T)
    if add is not None:
        exp = exp + add.double()
        size = size + add.double().abs()
    within(name, got, exp, 4 * step * size)


def make(T, d, f, dtype, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s, k=1.0: (torch.randn(s, generator=g, device="cuda") * k).to(dtype)  # noqa: E731
    return dict(x=r(T, d), wgu=r(2 * f, d, k=1.5 * d ** -0.5), wd=r(d, f, k=f ** -0.5), dy=r(T, d), add=r(T, d), dadd=r(T, d))


def check_forward(ffn, s, act, add):
    T, f, dt = ffn.T, ffn.f, ffn.dtype
    y = ffn.forward(s["x"], s["wgu"], s["wd"], add=s["add"] if add else None)
    x, w = s["x"].double(), s["wgu"].double()
    ab = x @ w.T
    K = x.shape[1]
    noise = 4 * ((K / 16 + 16) * 2.0 ** -23 if dt == BF else (K + 16) * 2.0 ** -24) * torch.sqrt((x * x) @ (w * w).T)
    a, b = ab[:, :f], ab[:, f:]
    g, dg = gate(a, act)
    within("h", ffn.h, g * b, (dg.abs() * b.abs() + 1e-2) * noise[:, :f] + g.abs() * noise[:, f:] + 1e-5 * (a * b).abs() + 1e-30)
    if ffn.keep:
        kept = act8_dequantize(ffn.ab, ffn.ab_scales, F32).double()
        top = ab.abs().view(T, -1, 32).amax(2).repeat_interleave(32, 1)
        # half a step of a code: 2^-4 of the value, 2^-10 of a scale that is at most max / 224
        assert ((kept - ab).abs() <= 2.0 ** -4 * ab.abs() + 2.0 ** -10 / 224 * top + 2 * noise).all()
    elif ffn.ab is not None:
        within("ab", ffn.ab, ab, noise)
    product("y", y, ffn.h, s["wd"], dt, s["add"] if add else None)
    assert ffn.status() == 0
    counters = 256 + PARTS + 128 + -(-T // 8192) * 128            # status, parts of cut tiles, pairs done, rows of tiles written
    assert ffn.ws[:counters if dt == BF else 256].count_nonzero() == 0
    return y


def check_backward(ffn, s, act, add):
    f, dt = ffn.f, ffn.dtype
    ab = (act8_dequantize(ffn.ab, ffn.ab_scales, F32) if ffn.keep else ffn.ab).double()
    a, b = ab[:, :f], ab[:, f:]
    g, dg = gate(a, act)
    res = ffn.backward(s["dy"], s["x"], s["wgu"], s["wd"], add=s["dadd"] if add else None)
    dy, wd = s["dy"].double(), s["wd"].double()
    dh, K = dy @ wd, dy.shape[1]
    noise = 4 * ((K / 16 + 16) * 2.0 ** -23 if dt == BF else (K + 16) * 2.0 ** -24) * torch.sqrt((dy * dy) @ (wd * wd))
    within("da", ffn.dab[:, :f], dh * b * dg, (b * dg).abs() * noise + 1e-5 * (dh * b).abs() * (1 + a.abs()) + 1e-30)
    within("db", ffn.dab[:, f:], dh * g, g.abs() * noise + 1e-5 * (dh * a).abs() + 1e-30)
    if ffn.keep:
        within("h again", ffn.h, g * b, 1e-5 * (a * b).abs() + 1e-30)
    product("dx", res["dx"], ffn.dab, s["wgu"].T, dt, s["dadd"] if add else None)
    product("dw_gate_up", res["dw_gate_up"], ffn.dab.T, s["x"].T, dt)
    product("dw_down", res["dw_down"], s["dy"].T, ffn.h.T, dt)
    assert ffn.status() == 0 and ffn.ws[:256 + PARTS + 128 if dt == BF else 256].count_nonzero() == 0
    return res


FEW = [(1, 64, 64), (1, 2048, 1024), (2, 8, 8), (3, 72, 40), (8, 520, 1000), (9, 256, 264), (17, 264, 136), (24, 256, 8192), (31, 1032, 4104),
       (33, 128, 72), (57, 2048, 512), (64, 512, 1000), (1, 4096, 8192), (9, 4096, 2744), (24, 4096, 8192), (26, 8192, 4104), (41, 2112, 9608),
       (64, 4032, 5000), (20, 1088, 1344), (33, 2048, 704), (64, 704, 2112), (1, 4096, 2752),
       (13, 4928, 2560), (16, 2048, 5120)]
MANY = [(65, 64, 64), (100, 8, 8), (127, 136, 72), (256, 256, 256), (257, 520, 264), (700, 1032, 328), (1000, 2048, 1024), (2500, 1024, 2048),
        (3000, 64, 4096), (515, 4096, 96), (256, 4096, 2048), (1300, 1024, 1088)]


@pytest.mark.parametrize("act,add", [("silu", True), ("gelu", False)])
@pytest.mark.parametrize("T,d,f", FEW + MANY)
def test_forward(T, d, f, act, add):
    check_forward(GatedFFN(T, d, f, act=act, backward=False), make(T, d, f, BF, T + d + f), act, add)


@pytest.mark.parametrize("keep", [None, "f8"])
@pytest.mark.parametrize("act,add", [("silu", True), ("gelu", False)])
@pytest.mark.parametrize("T,d,f", [(1, 64, 64), (5, 8, 32), (64, 200, 96)] + [m for m in MANY if m[2] % 32 == 0] + [(300, 72, 8192), (130, 8192, 2048), (234, 72, 6752), (2, 424, 3296),
                                                                            (4178, 112, 2048), (3000, 264, 896)])
def test_step(T, d, f, act, add, keep):
    s = make(T, d, f, BF, T + d + f)
    ffn = GatedFFN(T, d, f, act=act, keep=keep)
    check_forward(ffn, s, act, add)
    check_backward(ffn, s, act, add)


@pytest.mark.parametrize("T,d,f", [(7, 40, 8), (130, 136, 72), (700, 1032, 328)])
def test_step_narrow_features(T, d, f):
    s = make(T, d, f, BF, 1)
    ffn = GatedFFN(T, d, f)
    check_forward(ffn, s, "silu", False)
    check_backward(ffn, s, "silu", False)


@pytest.mark.parametrize("act,add", [("silu", True), ("gelu", False)])
@pytest.mark.parametrize("T,d,f", [(1, 1, 1), (3, 7, 5), (16, 64, 64), (203, 501, 337), (65, 1001, 130), (700, 300, 999), (2100, 513, 2050)])
def test_step_f32(T, d, f, act, add):
    s = make(T, d, f, F32, T + d + f)
    ffn = GatedFFN(T, d, f, F32, act=act)
    check_forward(ffn, s, act, add)
    check_backward(ffn, s, act, add)


def test_gradients_against_differences():
    T, d, f = 3, 20, 12
    for act in ("silu", "gelu"):
        s = make(T, d, f, F32, 4)
        ffn = GatedFFN(T, d, f, F32, act=act)
        ffn.forward(s["x"], s["wgu"], s["wd"])
        res = ffn.backward(s["dy"], s["x"], s["wgu"], s["wd"])

        def loss(x, wgu, wd):
            ab = x @ wgu.T
            return (((gate(ab[:, :f], act)[0] * ab[:, f:]) @ wd.T) * s["dy"].double()).sum()

        v = {k: s[k].double() for k in ("x", "wgu", "wd")}
        g = torch.Generator(device="cuda").manual_seed(9)
        for k, name in (("x", "dx"), ("wgu", "dw_gate_up"), ("wd", "dw_down")):
            u = torch.randn(v[k].shape, generator=g, device="cuda", dtype=torch.float64)
            h = 1e-5                                     # error of the difference: h^2, and 2^-52 of the loss over h
            diff = (loss(**{**v, k: v[k] + h * u}) - loss(**{**v, k: v[k] - h * u})) / (2 * h)
            grad = res[name].double()
            assert abs((grad * u).sum().item() - diff.item()) <= 1e-5 * (grad * u).abs().sum().item()


@pytest.mark.parametrize("T,dtype", [(1, BF), (40, BF), (300, BF), (50, F32)])
def test_in_place_and_repeatable(T, dtype):
    d, f = 264, 520
    s = make(T, d, f, dtype, 2)
    ffn, inf = GatedFFN(T, d, f, dtype), GatedFFN(T, d, f, dtype, backward=False)
    for blk in (ffn, inf):
        want = blk.forward(s["x"], s["wgu"], s["wd"], add=s["add"]).clone()
        room = torch.full((T + 4, d), 9.0, dtype=dtype, device="cuda")
        room[:T] = s["add"]
        assert blk.forward(s["x"], s["wgu"], s["wd"], add=room[:T], out=room[:T]).data_ptr() == room.data_ptr()
        assert torch.equal(room[:T], want) and room[T:].eq(9).all()
    ffn.forward(s["x"], s["wgu"], s["wd"])
    first = {k: v.clone() for k, v in ffn.backward(s["dy"], s["x"], s["wgu"], s["wd"], add=s["dadd"]).items()}
    ffn.dx.copy_(s["dadd"])
    again = ffn.backward(s["dy"], s["x"], s["wgu"], s["wd"], add=ffn.dx)
    assert all(torch.equal(first[k], again[k]) for k in first)


@pytest.mark.parametrize("keep", [None, "f8"])
@pytest.mark.parametrize("T", [3, 600])
def test_rows_that_are_not_finite(T, keep):
    """A NaN in one token: its rows of y and dx, and the weight gradients; no other token notices."""
    d, f = 256, 320
    s = make(T, d, f, BF, 3)
    bad = dict(s, x=s["x"].clone())
    bad["x"][1, 7] = float("nan")
    rest = [i for i in range(T) if i != 1]
    ffn, ref = GatedFFN(T, d, f, keep=keep), GatedFFN(T, d, f, keep=keep)
    y, want = ffn.forward(bad["x"], s["wgu"], s["wd"]), ref.forward(s["x"], s["wgu"], s["wd"])
    assert y[1].isnan().all() and torch.equal(y[rest], want[rest])
    a, b = ffn.backward(s["dy"], bad["x"], s["wgu"], s["wd"]), ref.backward(s["dy"], s["x"], s["wgu"], s["wd"])
    assert a["dx"][1].isnan().all() and torch.equal(a["dx"][rest], b["dx"][rest])
    assert a["dw_gate_up"].isnan().any() and a["dw_down"].isnan().any() and ffn.status() == 0
    few = GatedFFN(T, d, f, backward=False)
    y = few.forward(bad["x"], s["wgu"], s["wd"])
    assert y[1].isnan().all() and torch.isfinite(y[rest]).all()


def test_gate_at_large_arguments():
    """Projections in the hundreds and thousands: the sigmoid is 0 or 1, and nothing overflows on the way."""
    d = f = 64
    for act in ("silu", "gelu"):
        for T, dtype in ((3, BF), (80, BF), (5, F32)):
            s = make(T, d, f, dtype, 5)
            s["wgu"] = (s["wgu"].float() * 1000).to(dtype)
            ffn = GatedFFN(T, d, f, dtype, act=act)
            check_forward(ffn, s, act, False)
            check_backward(ffn, s, act, False)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_no_tokens(dtype):
    ffn = GatedFFN(0, 64, 32, dtype)
    s = make(0, 64, 32, dtype)
    ffn.dw_gate_up.fill_(3)
    ffn.dw_down.fill_(3)
    assert ffn.forward(s["x"], s["wgu"], s["wd"]).shape == (0, 64)
    res = ffn.backward(s["dy"], s["x"], s["wgu"], s["wd"])
    assert res["dw_gate_up"].eq(0).all() and res["dw_down"].eq(0).all() and res["dx"].shape == (0, 64)


@pytest.mark.parametrize("T", [1, 48, 333])
def test_stream_and_graph(T):
    d, f = 512, 768
    s = make(T, d, f, BF, 6)
    inf, ffn, ref = GatedFFN(T, d, f, backward=False), GatedFFN(T, d, f, keep="f8"), GatedFFN(T, d, f, keep="f8")

    def step(blk, x, stream=None):
        out = [inf.forward(x, s["wgu"], s["wd"], add=s["add"], stream=stream), blk.forward(x, s["wgu"], s["wd"], stream=stream)]
        return out + list(blk.backward(s["dy"], x, s["wgu"], s["wd"], stream=stream).values())

    want = [t.clone() for t in step(ref, s["x"])]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = step(ffn, s["x"], side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    x = s["x"].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(ffn, x)
    for k in range(3):                                    # the arrival counts are back at zero each time
        x.copy_(s["dy"] if k == 1 else s["x"])
        graph.replay()
        now = [t.clone() for t in got]
        assert all(torch.equal(a, b) for a, b in zip(now, step(ref, x)))


@pytest.mark.parametrize("T,d,f", [(1, 4096, 2744), (16, 4096, 2744), (24, 4096, 2744), (24, 4096, 4864), (60, 2048, 5120),
                                   (1, 4096, 2752), (16, 4096, 4864), (12, 4928, 2560)])
def test_repeats_with_weights_in_the_cache(T, d, f):
    """The ring of streamed weights turns fastest when nothing comes from memory: every pass gives the first one's bits."""
    s = make(T, d, f, BF, 7)
    ffn = GatedFFN(T, d, f, backward=False)
    first = check_forward(ffn, s, "silu", True).clone(), ffn.h.clone()
    for _ in range(30):
        ffn.h.fill_(7.0)
        assert torch.equal(ffn.forward(s["x"], s["wgu"], s["wd"], add=s["add"]), first[0]) and torch.equal(ffn.h, first[1])


def test_shared_scratch():
    T, d, f = 200, 128, 256
    scratch = dict(h=torch.empty(T, f, dtype=BF, device="cuda"), dab=torch.empty(T, 2 * f, dtype=BF, device="cuda"))
    s = [make(T, d, f, BF, i) for i in range(2)]
    shared, own = [GatedFFN(T, d, f, keep="f8", scratch=scratch) for _ in range(2)], [GatedFFN(T, d, f, keep="f8") for _ in range(2)]
    for blk in (shared, own):
        for b, v in zip(blk, s):
            b.forward(v["x"], v["wgu"], v["wd"])
    for b, o, v in list(zip(shared, own, s))[::-1]:
        p, q = b.backward(v["dy"], v["x"], v["wgu"], v["wd"]), o.backward(v["dy"], v["x"], v["wgu"], v["wd"])
        assert all(torch.equal(p[k], q[k]) for k in p)
    with pytest.raises(ValueError, match="shared"):
        GatedFFN(T, d, f, scratch=scratch)
    with pytest.raises(ValueError, match="scratch"):      # not where the block is
        GatedFFN(T, d, f, keep="f8", scratch={k: v.cpu() for k, v in scratch.items()})
