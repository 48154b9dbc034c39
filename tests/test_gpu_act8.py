"""Activations in 8 bits (moe_act8_*) against the format's definition: codes and scales bit for bit, since a division by a power
of two is exact and rounding to nearest even leaves nothing open."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from mixture_experts_layer_histogram_gb300 import act8_dequantize, act8_quantize
    from mixture_experts_layer_histogram_gb300 import _lib as L


def defined(x):
    """codes [R, K], scale bytes [R, blocks] and values (64 bits) of x [R, K]."""
    R, K = x.shape
    nb = -(-K // 32)
    b = torch.zeros(R, nb * 32, dtype=torch.float64, device=x.device)
    b[:, :K] = x.double()
    b = b.view(R, nb, 32)
    top = b.abs().amax(2)
    byte = torch.zeros(R, nb, dtype=torch.int64, device=x.device)
    for e in range(-126, 130):                        # the least power that is enough, by trying every one
        byte += (448 * 2.0 ** (e - 1) < top).long()
    bad = ~torch.isfinite(b).all(2)
    byte[bad] = 255
    scale = torch.exp2(byte.double() - 127)
    y = torch.where(bad[..., None], torch.zeros_like(b), b / scale[..., None])
    codes = y.float().to(torch.float8_e4m3fn)         # y is exact in fp32 (a power of two times x), the cast rounds to even
    v = codes.double() * torch.where(bad, torch.full_like(scale, float("nan")), scale)[..., None]
    return codes.view(torch.uint8).view(R, -1)[:, :K], byte, v.view(R, -1)[:, :K]


def check(x):
    codes, scales = act8_quantize(x)
    ec, es, ev = defined(x)
    assert torch.equal(codes, ec)
    assert torch.equal(scales.view(es.shape).long(), es)
    for dtype in (torch.float32, torch.bfloat16):
        v = act8_dequantize(codes, scales, dtype)
        assert torch.equal(v.isnan(), ev.isnan())
        assert torch.equal(v.nan_to_num(0.0), ev.float().to(dtype).nan_to_num(0.0))
    return ev


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("R,K", [(1, 1), (1, 32), (3, 31), (2, 33), (5, 16), (7, 48), (1, 4096), (129, 96), (77, 999), (513, 1024)])
def test_random(R, K, dtype):
    g = torch.Generator(device="cuda").manual_seed(R * 7 + K)
    x = torch.randn(R, K, generator=g, device="cuda") * torch.exp(8 * torch.randn(R, K, generator=g, device="cuda").round())
    ev = check(x.to(dtype))
    x = x.to(dtype).double()
    # half a step of the code: 2^-4 of the value, or of 2^-6 of the scale where the code is subnormal
    assert ((ev - x).abs() <= 2.0 ** -4 * x.abs() + 2.0 ** -10 * torch.exp2(defined(x.float())[1].double() - 127).repeat_interleave(32, 1)[:, :K]).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("K", [64, 40])
def test_borders(K, dtype):
    rows = []
    for top in (0.0, 448.0, 449.0, 450.0, 447.0, 1.75, 1.7578125, 1.75 * 2.0 ** 120, 3.0e38, 2.0 ** -126, 2.0 ** -133, 1.75 * 2.0 ** -118,
                1.78 * 2.0 ** -118, float("inf"), float("-inf"), float("nan")):
        r = torch.zeros(K)
        r[3], r[7], r[K - 1] = top, -top / 3, top / 64
        rows.append(r)
        r = torch.linspace(-1, 1, K) * (top if abs(top) < 1e39 else 1.0)
        r[K // 2] = top
        rows.append(r)
    ties = torch.arange(K).float() * 0.0625 + 1.0 + 0.0625       # half-way between neighbours of e4m3
    ties[0] = 448.0
    rows.append(ties)
    check(torch.stack(rows).to(dtype).cuda())


def test_nan_stays_in_its_block():
    x = torch.ones(2, 96, device="cuda")
    x[0, 40] = float("nan")
    x[1, 95] = float("inf")
    v = act8_dequantize(*act8_quantize(x), torch.float32)
    assert v[0, 32:64].isnan().all() and v[1, 64:].isnan().all() and v.isnan().sum() == 64 and (v[~v.isnan()] == 1).all()


def test_no_rows_and_leading_dimensions():
    codes, scales = act8_quantize(torch.empty(0, 64, device="cuda"))
    assert codes.shape == (0, 64) and scales.numel() == 0 and act8_dequantize(codes, scales).shape == (0, 64)
    x = torch.randn(3, 5, 40, device="cuda")
    codes, scales = act8_quantize(x)
    assert torch.equal(codes.view(15, 40), act8_quantize(x.view(15, 40))[0])
    out = torch.empty_like(x)
    assert act8_dequantize(codes, scales, torch.float32, out=out) is out


@pytest.mark.parametrize("K", [4096, 4100])
def test_offsets_past_32_bits(K):
    R = 2 ** 31 // 2048 + 9                         # twice 2^31 values: offsets pass 32 bits
    x = torch.empty(R, K, dtype=torch.bfloat16, device="cuda")
    x.normal_(generator=torch.Generator(device="cuda").manual_seed(1))
    codes, scales = act8_quantize(x)
    v = act8_dequantize(codes, scales)
    for rows in (slice(0, 3), slice(R // 2 - 2, R // 2 + 2), slice(R - 3, R)):
        ec, es, ev = defined(x[rows])
        assert torch.equal(codes[rows], ec) and torch.equal(scales.view(R, -1)[rows].long(), es) and torch.equal(v[rows], ev.bfloat16())


def test_stream_and_graph():
    x = torch.randn(64, 256, device="cuda").bfloat16()
    codes, scales = torch.empty(64, 256, dtype=torch.uint8, device="cuda"), torch.empty(64 * 8, dtype=torch.uint8, device="cuda")
    out = torch.empty_like(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    L.moe_act8_quantize(x, codes, scales, stream=side)
    L.moe_act8_dequantize(codes, scales, out, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out.double(), defined(x)[2])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        L.moe_act8_quantize(x, codes, scales)
        L.moe_act8_dequantize(codes, scales, out)
    x.copy_(torch.randn(64, 256, device="cuda"))
    graph.replay()
    assert torch.equal(out.double(), defined(x)[2])
