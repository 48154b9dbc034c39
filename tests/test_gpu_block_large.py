"""Sizes whose offsets pass 32 bits: the tail of a tensor of more than 2^31 values is what it is on a small copy of it."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from mixture_experts_layer_histogram_gb300 import AdamW, BlockNorms, fp4_dequantize, fp4_quantize


@pytest.fixture(autouse=True)
def release():
    yield
    torch.cuda.empty_cache()


def test_norms_past_2_31_values():
    T, d, tail = 600_000, 4096, 64
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.empty((T, d), dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    y = torch.empty_like(x).normal_(generator=g)
    w = (1 + 0.1 * torch.randn(d, generator=g, device="cuda")).bfloat16()
    big = BlockNorms(T, d, gate="channel", res_scale=0.5)
    small = BlockNorms(tail, d, gate="channel", res_scale=0.5)
    out, n = big.post(y, x, w, gate=w, w_next=w)
    o2, n2 = small.post(y[-tail:].clone(), x[-tail:].clone(), w, gate=w, w_next=w)
    assert torch.equal(out[-tail:], o2) and torch.equal(n[-tail:], n2)
    res = big.post_backward(x, y, out, y, w, gate=w, w_next=w)
    r2 = small.post_backward(x[-tail:].clone(), y[-tail:].clone(), o2, y[-tail:].clone(), w, gate=w, w_next=w)
    assert torch.equal(res["dx"][-tail:], r2["dx"]) and torch.equal(res["dy"][-tail:], r2["dy"])


@pytest.mark.parametrize("state", ["f32", "f8"])
def test_adamw_past_2_31_values(state):
    n, tail = (1 << 31) + 4096 + 100, 4096 + 100
    g = torch.Generator(device="cuda").manual_seed(2)
    p = torch.empty(n, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    q = torch.empty(n, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    master = p[-tail:].clone().float()
    ps, qs = p[-tail:].clone(), q[-tail:].clone()
    big = AdamW([p], [q], lr=1e-2, state=state)
    big.step()
    small = AdamW([ps], [qs], lr=1e-2, state=state)
    small.step()
    m, v = big.m[0][-tail:].float(), big.v[0][-tail:].float()
    if state == "f32":
        assert torch.equal(m, small.m[0]) and torch.equal(v, small.v[0])
    else:   # the dither differs (the place enters it): codes one step apart at most, scales the same
        assert torch.equal(big.m_scale[0][-17:], small.m_scale[0])
        assert ((m - small.m[0].float()).abs() <= 0.1251 * m.abs().clamp_min(2.0 ** -6)).all()
    assert ((p[-tail:].float() - ps.float()).abs() <= 2.0 ** -7 * ps.float().abs() + 1e-30).all()
    assert ((p[-tail:].float() - master).abs() > 0).any()


def test_quantisation_in_several_launches():
    """2^31 vectors of sixteen values (rows padded to 128) are more than one launch counts."""
    R, K = (1 << 28) + 300, 32
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.empty((R, K), dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    codes, scales = fp4_quantize(x)
    back = fp4_dequantize(codes, scales)
    for lo, hi in ((0, 256), ((1 << 28) - 512, (1 << 28) + 300)):
        lo -= lo % 128
        c2, s2 = fp4_quantize(x[lo:hi].clone())
        assert torch.equal(codes[lo:hi], c2) and torch.equal(scales[lo // 128 * 512:lo // 128 * 512 + s2.numel()], s2)
        assert torch.equal(back[lo:hi], fp4_dequantize(c2, s2))
