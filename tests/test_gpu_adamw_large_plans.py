"""Plans of more chunks than the GPU runs at once, for every kind of tensor: blocks take several chunks, whole ones, a
ragged one and those of a tensor off the 16-byte grid. And the parameter of every kind with 8-bit states.

Tolerances are those of test_gpu_adamw.py: fp32 values 2e-6 of the tensor's largest magnitude; values in few bits within
one step of the exact value, and 2e-4 of them on the other side of a rounding threshold. A bf16 parameter is the fp32 result
p0 + change rounded within one of its steps. That result is off by `delta`: 2^-20 of the change (some sixteen roundings,
approximations and constants of 2^-24 each) and 2^-22 of p0; where the two all but cancel, delta is not small
against the step of what is left (millions of values hold such ones), so it stands beside the step.
"""
import pytest
import torch

from test_gpu_adamw import HY, SIZES, blocks, e4m3_down, step64, weyl, within

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from mixture_experts_layer_histogram_gb300 import AdamW

KINDS = [(torch.float32, False), (torch.bfloat16, False), (torch.bfloat16, True)]
LARGE = [4_200_001, 1_000_003, 300_000]      # the second starts off the 16-byte grid


def tensors(sizes, dtype, scale, gen):
    out = []
    for i, n in enumerate(sizes):
        skip = 1 if n == LARGE[1] else 0
        out.append((torch.randn(n + skip, generator=gen, device="cuda") * scale).to(dtype)[skip:])
    return out


def held64(opt, i, n):
    if opt.state == "f32":
        return opt.m[i].double(), opt.v[i].double()
    ms, vs = (s[i].double().repeat_interleave(256)[:n] for s in (opt.m_scale, opt.v_scale))
    return opt.m[i].double() * ms, (opt.v[i].double() * vs) ** 2


def check_codes(opt, i, name, val, t, shift):
    n = val.numel()
    pad = torch.zeros(blocks(n) * 256, dtype=torch.float64, device="cuda")
    pad[:n] = val.abs()
    scale = pad.view(-1, 256).amax(1) / 448
    within(getattr(opt, name + "_scale")[i], scale)
    u = torch.div(weyl(n, t, shift), 4096, rounding_mode="floor").double()
    y = torch.where(scale > 0, 1 / scale, 0.0).repeat_interleave(256)[:n] * val.abs()
    got = getattr(opt, name)[i].double()
    assert (got != torch.sign(val) * e4m3_down(y, u)).sum().item() <= max(1, 2e-4 * n), (name, n, t)
    step = torch.exp2(torch.floor(torch.log2(y.clamp_min(2.0 ** -6))) - 3)
    assert ((got - torch.sign(val) * y).abs() <= step * 1.0001).all(), (name, n, t)


def step_of(x):
    return torch.exp2(torch.floor(torch.log2(x.abs().clamp_min(2.0 ** -126))) - 7)


def check_dithered(p, p0, x, t):
    u = torch.div(weyl(p.numel(), t, 0xAAAAAAAA), 65536, rounding_mode="floor").double() / 65536
    delta = 2.0 ** -20 * (x - p0).abs() + 2.0 ** -22 * p0.abs()
    assert ((p.double() - x).abs() <= step_of(x.abs() + delta) + delta).all()
    ulp = step_of(x)
    assert (p.double() != torch.sign(x) * torch.floor(x.abs() / ulp + u) * ulp).sum().item() <= max(1, 2e-4 * p.numel())


@pytest.mark.parametrize("sizes", [LARGE, SIZES], ids=["large", "small"])
@pytest.mark.parametrize("state", ["f32", "f8"])
@pytest.mark.parametrize("dtype,master", KINDS)
def test_every_kind(dtype, master, state, sizes):
    gen = torch.Generator(device="cuda").manual_seed(11)
    ps, gs = tensors(sizes, dtype, 0.05, gen), tensors(sizes, dtype, 1e-2, gen)
    wds = [0.1 if i % 2 == 0 else 0.0 for i in range(len(sizes))]
    masters = [torch.empty(p.numel() + 1, device="cuda")[p.numel() & 1:][:p.numel()].copy_(p) for p in ps] if master else None
    opt = AdamW(ps, gs, weight_decay=wds, state=state, masters=masters, **HY)
    for t in range(1, 4):
        start = [(opt.masters[i] if master else p).double() for i, p in enumerate(ps)]
        held = [held64(opt, i, p.numel()) for i, p in enumerate(ps)]
        opt.step()
        for i, p in enumerate(ps):
            x, m, v = step64(start[i], gs[i], *held[i], t, wds[i])
            if state == "f32":
                within(opt.m[i], m)
                within(opt.v[i], v)
            else:
                check_codes(opt, i, "m", m, t, 0)
                check_codes(opt, i, "v", v.sqrt(), t, 0x55555555)
            if master:
                within(opt.masters[i], x)
                assert torch.equal(p, opt.masters[i].to(torch.bfloat16))
            elif dtype == torch.float32:
                within(p, x)
            else:
                check_dithered(p, start[i], x, t)
        for q in gs:
            q.copy_((torch.randn(q.shape, generator=gen, device="cuda") * 1e-2).to(dtype))
    assert opt.steps == 3
