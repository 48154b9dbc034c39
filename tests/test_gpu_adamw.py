"""AdamW (moe_adamw_*, AdamW) against the formulas in 64 bits.

Tolerances. fp32 states and parameters: a step rounds a handful of times (2^-24 each) and five steps are taken, so
2e-6 of the tensor's largest magnitude bounds them. Codes in few bits: the fp32 value in front of the rounding is off by
a few 2^-24, so it falls on the other side of a rounding threshold for about 2 * 4 * 2^-24 * 16 = 8e-6 of the
values; 2e-4 may differ (small tensors: one value), and by one code only.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from mixture_experts_layer_histogram_gb300 import AdamW
    from mixture_experts_layer_histogram_gb300 import _lib as L

HY = dict(lr=1e-3, betas=(0.9, 0.99), eps=1e-8)
SIZES = [1, 7, 8, 255, 256, 257, 2047, 2048, 4096, 4097, 12345, 1 << 17]


def blocks(n):
    return -(-n // 256)


def step64(p, g, m, v, t, wd, scale=1.0):
    b1, b2 = HY["betas"]
    g = g.double() * scale
    m = b1 * m.double() + (1 - b1) * g
    v = b2 * v.double() + (1 - b2) * g * g
    p = p.double() * (1 - HY["lr"] * wd) - HY["lr"] * (m / (1 - b1 ** t)) / (torch.sqrt(v / (1 - b2 ** t)) + HY["eps"])
    return p, m, v


def within(got, exp, tol=2e-6):
    top = exp.abs().max().item()
    assert (got.double() - exp).abs().max().item() <= tol * top + 1e-30


def weyl(n, t, shift):
    i = torch.arange(n, dtype=torch.int64, device="cuda")
    return (i * 2654435769 + t * 1640531535 + shift) % (1 << 32)


def e4m3_down(y, u20):
    """y >= 0 (float64) rounded down on the e4m3 grid after adding u20 / 2^20 of a step."""
    e = torch.floor(torch.log2(y.clamp_min(2.0 ** -6)))
    ulp = torch.exp2(e - 3)
    return (torch.floor(y / ulp + u20 / 2.0 ** 20) * ulp).clamp_max(448.0)


@pytest.mark.parametrize("dtype,master", [(torch.float32, False), (torch.bfloat16, False), (torch.bfloat16, True)])
def test_fp32_states(dtype, master):
    g = torch.Generator().manual_seed(3)
    ps = [torch.randn(n, generator=g).mul(0.05).to(dtype).cuda() for n in SIZES]
    gs = [torch.randn(n, generator=g).mul(1e-2).to(dtype).cuda() for n in SIZES]
    wds = [0.1 if i % 2 else 0.0 for i in range(len(SIZES))]
    opt = AdamW(ps, gs, weight_decay=wds, masters=True if master else None, **HY)
    ref = [(p.double(), torch.zeros(p.shape, device="cuda").double(), torch.zeros(p.shape, device="cuda").double())
           for p in ps]
    for t in range(1, 6):
        for q in gs:
            q.copy_((torch.randn(q.shape, generator=g) * 1e-2).to(dtype))
        before = [p.clone() for p in ps]
        opt.step()
        for i, (p, q) in enumerate(zip(ps, gs)):
            start = ref[i][0] if master or dtype == torch.float32 else before[i]
            ref[i] = step64(start, q, ref[i][1], ref[i][2], t, wds[i])
            within(opt.m[i], ref[i][1])
            within(opt.v[i], ref[i][2])
            if master:
                within(opt.masters[i], ref[i][0])
                assert torch.equal(p, opt.masters[i].to(torch.bfloat16))
            elif dtype == torch.float32:
                within(p, ref[i][0])
            else:   # dithered: one of the two neighbours of the exact value, the one the sequence picks
                u = torch.div(weyl(p.numel(), t, 0xAAAAAAAA), 65536, rounding_mode="floor").double() / 65536
                x = ref[i][0]
                ulp = torch.exp2(torch.floor(torch.log2(x.abs().clamp_min(2.0 ** -126))) - 7)
                exp = torch.sign(x) * torch.floor(x.abs() / ulp + u) * ulp
                assert ((p.double() - x).abs() <= ulp * (1 + 1e-4)).all()
                assert (p.double() != exp).sum().item() <= max(1, 2e-4 * p.numel())
    assert opt.steps == 5


@pytest.mark.parametrize("dtype,master", [(torch.float32, False), (torch.bfloat16, False), (torch.bfloat16, True)])
def test_8bit_states(dtype, master):
    g = torch.Generator().manual_seed(4)
    ps = [torch.randn(n, generator=g).mul(0.05).to(dtype).cuda() for n in SIZES]
    gs = [torch.randn(n, generator=g).mul(1e-2).to(dtype).cuda() for n in SIZES]
    opt = AdamW(ps, gs, weight_decay=0.1, state="f8", masters=True if master else None, **HY)
    for t in range(1, 5):
        start = [(opt.masters[i] if master else p).double() for i, p in enumerate(ps)]
        held = []
        for i, p in enumerate(ps):
            n = p.numel()
            ms, vs = (s[i].double().repeat_interleave(256)[:n] for s in (opt.m_scale, opt.v_scale))
            held.append((opt.m[i].double() * ms, (opt.v[i].double() * vs) ** 2))
        opt.step()
        for i, p in enumerate(ps):
            n = p.numel()
            x, m, v = step64(start[i], gs[i], held[i][0], held[i][1], t, 0.1)
            if master:
                within(opt.masters[i], x)
            elif dtype == torch.float32:
                within(p, x)
            for name, val, shift in (("m", m, 0), ("v", v.sqrt(), 0x55555555)):
                pad = torch.zeros(blocks(n) * 256, dtype=torch.float64, device="cuda")
                pad[:n] = val.abs()
                scale = pad.view(-1, 256).amax(1) / 448
                got_scale = getattr(opt, name + "_scale")[i]
                within(got_scale, scale)
                u = torch.div(weyl(n, t, shift), 4096, rounding_mode="floor").double()
                y = torch.where(scale > 0, 1 / scale, 0.0).repeat_interleave(256)[:n] * val.abs()
                exp = torch.sign(val) * e4m3_down(y, u)
                got = getattr(opt, name)[i].double()
                bad = got != exp
                assert bad.sum().item() <= max(1, 2e-4 * n), (name, n, bad.sum().item())
                step = torch.exp2(torch.floor(torch.log2(y.clamp_min(2.0 ** -6))) - 3)
                assert ((got - torch.sign(val) * y).abs() <= step * 1.0001).all()
        for q in gs:
            q.copy_((torch.randn(q.shape, generator=g) * 1e-2).to(dtype))


def test_8bit_second_moment_follows_slow_changes():
    """beta2 = 0.999 moves sqrt(v) by a fraction of an e4m3 step per step of the optimiser. From v of (1e-2)^2 under
    gradients of 1e-3 times a factor of 0.6..1.4 per element, v after 2000 steps is known. A value sits within
    one code (12.5 %) of its place, both ways alike, so the mean over 8192 elements lies within 2 %; rounding to
    nearest would leave it at its start, nine times higher."""
    n = 8192
    k = (0.6 + 0.8 * torch.arange(n, device="cuda") / n)[torch.randperm(n, generator=torch.Generator().manual_seed(0)).cuda()]
    p = torch.zeros(n, device="cuda")
    g = 1e-3 * k
    root = 1e-2 * k
    scale = root.view(-1, 256).amax(1) / 448
    v = (root.view(-1, 256) / scale[:, None]).to(torch.float8_e4m3fn).view(-1)
    opt = AdamW([p], [g], lr=0.0, betas=(0.9, 0.999), state="f8", m=[torch.zeros(n, device="cuda").to(torch.float8_e4m3fn)],
                v=[v], m_scale=[torch.zeros(n // 256, device="cuda")], v_scale=[scale])
    for _ in range(2000):
        opt.step()
    keep = 0.999 ** 2000
    exp = torch.sqrt(keep * root.double() ** 2 + (1 - keep) * g.double() ** 2)
    got = opt.v[0].double() * opt.v_scale[0].double().repeat_interleave(256)
    assert abs((got / exp).mean().item() - 1) <= 0.02


def test_mixed_kinds_unaligned_views_and_other_stream():
    """fp32 and bf16 tensors in one plan, views that start off the 16-byte grid, and the launch on another stream."""
    flat = torch.randn(5000, device="cuda") * 0.05
    half = (torch.randn(5000, device="cuda") * 0.05).bfloat16()
    ps = [flat[1:1000], half[3:2000], flat[1003:1003], flat[2001:5000]]
    gs = [torch.randn(p.numel() + 1, device="cuda").to(p.dtype)[1:] * 1e-2 for p in ps]
    gs = [torch.empty(g.numel() + 1, device="cuda", dtype=g.dtype)[1:].copy_(g) for g in gs]
    keep_flat, keep_half = flat.clone(), half.clone()
    start = [p.double() for p in ps]
    opt = AdamW(ps, gs, weight_decay=0.0, **HY)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    opt.step(stream=side)
    torch.cuda.synchronize()
    for i in (0, 3):
        x, m, v = step64(start[i], gs[i], torch.zeros_like(start[i]), torch.zeros_like(start[i]), 1, 0.0)
        within(ps[i], x)
        within(opt.m[i], m)
    x, m, _ = step64(start[1], gs[1], torch.zeros_like(start[1]), torch.zeros_like(start[1]), 1, 0.0)
    within(opt.m[1], m)
    assert ((ps[1].double() - x).abs() <= 2.0 ** -7 * x.abs() + 1e-30).all()
    for a, b, spans in ((flat, keep_flat, [(0, 1), (1000, 2001)]), (half, keep_half, [(0, 3), (2000, 5000)])):
        for lo, hi in spans:    # nothing outside the views is written
            assert torch.equal(a[lo:hi], b[lo:hi])
    assert opt.steps == 1


def test_gradient_scale_lr_and_graph_replay():
    p = torch.randn(4000, device="cuda")
    g = torch.randn(4000, device="cuda")
    opt = AdamW([p], [g], weight_decay=0.0, **HY)
    ref = (p.double(), torch.zeros(4000, device="cuda").double(), torch.zeros(4000, device="cuda").double())
    opt.step()
    ref = step64(*[ref[0], g, ref[1], ref[2]], 1, 0.0)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        opt.step()
    assert opt.steps == 1
    opt.set_grad_scale(0.5)
    for t in (2, 3):
        graph.replay()
        ref = step64(ref[0], g, ref[1], ref[2], t, 0.0, scale=0.5)
    assert opt.steps == 3
    within(p, ref[0])
    within(opt.v[0], ref[2])
    opt.set_lr(0.0)
    before = p.clone()
    graph.replay()
    assert torch.equal(p, before)


def test_empty_plan_counts_and_non_finite_gradients_stay_local():
    opt = AdamW([], [], **HY)
    opt.step()
    assert opt.steps == 1
    for state in ("f32", "f8"):
        p = torch.ones(1024, device="cuda")
        g = torch.full((1024,), 1e-2, device="cuda")
        g[300] = float("nan")
        opt = AdamW([p], [g], state=state, **HY)
        opt.step()
        bad = ~torch.isfinite(p)
        assert bad.nonzero().view(-1).tolist() == [300]
        m = opt.m[0].float()
        assert torch.isnan(m).nonzero().view(-1).tolist() == [300]


def test_refusals():
    p, g = torch.zeros(64, device="cuda"), torch.zeros(64, device="cuda")
    with pytest.raises(ValueError):
        AdamW([p], [])
    with pytest.raises(ValueError):
        AdamW([p], [g], state="int8")
    with pytest.raises(ValueError):
        AdamW([p], [g.bfloat16()])
    with pytest.raises(ValueError):
        AdamW([p.view(8, 8).t()], [g.view(8, 8)])
    with pytest.raises(ValueError):
        AdamW([p.cpu()], [g.cpu()])
    with pytest.raises(ValueError):
        AdamW([p], [g], state="f8", m=[torch.zeros(64, device="cuda")])
    with pytest.raises(ValueError):
        AdamW([p], [g], weight_decay=[0.1, 0.1])
    with pytest.raises(L.MoeError):
        AdamW([p], [g], weight_decay=-1.0)
    with pytest.raises(L.MoeError):
        AdamW([p], [g], masters=[p.clone()])                  # a master copy of an fp32 parameter
    with pytest.raises(L.MoeError):
        AdamW([p], [g], betas=(1.0, 0.9)).step()
    assert math.isfinite(p.sum().item())


def test_subnormal_second_moment():
    """Gradients of 1e-19 and an eps below them: v is about 1e-40, held in steps of 2^-149, so its root is off by at most
    2^-150 / 1e-40 / 2 = 4e-6 and the update, lr in size, by that and a few 2^-22 (approximate root and
    reciprocal): 1e-5."""
    n = 5000
    k = 1 + torch.arange(n, device="cuda") / n
    p, g = torch.zeros(n, device="cuda"), 1e-19 * k
    opt = AdamW([p], [g], lr=1e-3, betas=(0.9, 0.99), eps=1e-30, weight_decay=0.0)
    opt.step()
    m, v = 0.1 * g.double(), 0.01 * g.double() ** 2
    exp = -1e-3 * (m / 0.1) / (torch.sqrt(v / 0.01) + 1e-30)
    assert ((p.double() - exp).abs() <= 1e-5 * 1e-3).all()


def test_refusals_of_masters_and_eps():
    p = torch.zeros(64, device="cuda", dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        AdamW([p, p.clone()], [p.clone(), p.clone()], masters=[p.float()])
    with pytest.raises(L.MoeError):
        AdamW([p], [p.clone()], eps=1e-40).step()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_8bit_codes_bit_for_bit(dtype):
    """8-bit states of fp32 parameters, or of bf16 ones with a master: codes and scales are those of the formulas in
    fp32, each operation rounded to nearest, over 20 steps and 1.3 million values. (The scale's inverse is the rounded
    reciprocal of the largest magnitude times 448; below the smallest normal code what lies below 2^-20 of a step is
    dropped.) Gradients span six orders of magnitude, so codes near zero, where one step matters most, are among them."""
    n = 256 * 5000 + 100
    gen = torch.Generator(device="cuda").manual_seed(8)
    wide = torch.pow(10.0, -6 * torch.rand(n, generator=gen, device="cuda"))
    p = (torch.randn(n, generator=gen, device="cuda") * 0.02).to(dtype)
    grad = torch.empty(n, device="cuda", dtype=dtype)
    opt = AdamW([p], [grad], state="f8", masters=True if dtype == torch.bfloat16 else None, **HY)
    f32 = dict(dtype=torch.float32, device="cuda")
    nb = blocks(n)
    m, v = torch.zeros(nb, 256, **f32), torch.zeros(nb, 256, **f32)
    ms, vs = torch.zeros(nb, 1, **f32), torch.zeros(nb, 1, **f32)
    b1, b2 = HY["betas"]

    def codes(val, t, shift):
        top = val.abs().amax(1, keepdim=True)
        keep = top >= 1e-30
        y = (val * torch.where(keep, torch.reciprocal(top) * 448.0, 0.0)).abs()
        u = torch.div(weyl(n, t, shift), 4096, rounding_mode="floor").int()
        u = torch.nn.functional.pad(u, (0, nb * 256 - n)).view(nb, 256)
        normal = ((y.view(torch.int32) + u) & -(1 << 20)).view(torch.float32)
        small = (((y * 2.0 ** 29).int() + u) >> 20).float() * 2.0 ** -9
        code = torch.where(y < 2.0 ** -6, small, normal).clamp_max(448.0)
        return torch.where(val < 0, -code, code), torch.where(keep, top * (1.0 / 448.0), 0.0), torch.where(keep, top / 448.0, 0.0)

    for t in range(1, 21):
        grad.copy_((torch.randn(n, generator=gen, device="cuda") * wide).to(dtype))
        g = torch.nn.functional.pad(grad.float(), (0, nb * 256 - n)).view(nb, 256)
        opt.step()
        a = v * vs
        m, v = b1 * (m * ms) + (1 - b1) * g, b2 * (a * a) + (1 - b2) * (g * g)
        (m, ms, ms2), (v, vs, vs2) = codes(m, t, 0), codes(v.sqrt(), t, 0x55555555)
        for got, exp in ((opt.m[0].float(), m), (opt.v[0].float(), v)):
            assert torch.equal(got, exp.view(-1)[:n]), t
        for got, exp, other in ((opt.m_scale[0], ms, ms2), (opt.v_scale[0], vs, vs2)):
            assert torch.equal(got, exp.view(-1)) or torch.equal(got, other.view(-1))
        ms, vs = opt.m_scale[0].view(-1, 1).clone(), opt.v_scale[0].view(-1, 1).clone()
