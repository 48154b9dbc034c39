"""Weight decay where lr * weight_decay is small (the tail of a schedule).

With gradients and states of zero a step is p' = p (1 - lr wd) alone. The kernel forms lr wd in fp32 (off by 2^-24 of
itself beyond the rounding of the two factors, which the reference takes as fp32 too), their product with p, and the sum:
p' is within half a step of fp32, plus 2^-22 of the change, of the 64-bit value.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from mixture_experts_layer_histogram_gb300 import AdamW

N = 70_001


def f32(x):
    return torch.tensor(x, dtype=torch.float32).double().item()


def ulp32(x):
    return torch.exp2(torch.floor(torch.log2(x.abs())) - 23)


@pytest.mark.parametrize("state", ["f32", "f8"])
@pytest.mark.parametrize("kind", ["f32", "master", "bf16"])
@pytest.mark.parametrize("lr,wd", [(1e-4, 0.01), (1e-5, 0.01), (5e-6, 0.01), (1e-3, 0.1)])
def test_small_decay(lr, wd, kind, state):
    g = torch.Generator(device="cuda").manual_seed(6)
    p = torch.randn(N, generator=g, device="cuda") * 3
    p = torch.where(p.abs() < 1e-6, 1.0, p)
    p = p if kind == "f32" else p.bfloat16()
    start = p.double()
    opt = AdamW([p], [torch.zeros_like(p)], lr=lr, weight_decay=wd, state=state, masters=True if kind == "master" else None)
    opt.step()
    change = f32(lr) * f32(wd) * start
    exp = start - change
    bound = 0.5 * ulp32(start) * (1 + 2.0 ** -20) + 2.0 ** -22 * change.abs()
    if kind != "bf16":
        got = (p if kind == "f32" else opt.masters[0]).double()
        assert ((got - exp).abs() <= bound).all()
        return
    # without a master: that value, rounded down after adding u / 2^16 of a step. Its last bit changes the result
    # for 1 in 2^16 values, twice that is allowed for (and a few more).
    i = torch.arange(N, device="cuda")
    u = torch.div((i * 2654435769 + 1640531535 + 0xAAAAAAAA) % (1 << 32), 65536, rounding_mode="floor").int()
    want = ((exp.float().view(torch.int32) + u) & -65536).view(torch.float32)
    assert (p.float() != want).sum().item() <= 2 + 4 * N // 65536
