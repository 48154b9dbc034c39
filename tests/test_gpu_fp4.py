"""MXFP4: quantisation, reading back, the quantising permutation, and the grouped FFN on 4-bit operands.

Quantisation divides by a power of two and rounds to nearest even, both exact to define, so codes and values are
compared with ==. The FFN is checked in two halves. h: the fp32 value in front of the rounding is off from the 64-bit one
by at most about 1e-5 of its block's largest value (fp32 sums of up to 2048 products, the approximate sigmoid), so
about 2 * 1e-5 / (1/12) = 2e-4 of the values can fall on the other side of a rounding threshold (2e-3 allowed), and by
one step of the grid. y: from the h codes that the kernel wrote, bf16 rounding (2^-8 relative) and 2e-5 of the largest |y|.
"""
import pytest
import torch

import moe_inputs
import oracle

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from mixture_experts_layer_histogram_gb300 import Fp4Weights, MoELayerFp4, fp4_dequantize, fp4_quantize
    from mixture_experts_layer_histogram_gb300 import _lib as L

GRID = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64)


def mx64(x):
    """Codes (0..15) and scale exponents of x [R, K] from the definition, on the CPU in 64 bits."""
    b = x.double().cpu().view(x.shape[0], -1, 32)
    top = b.abs().amax(2)
    _, e = torch.frexp(top)
    e = torch.where(top > 0, e - 3, torch.full_like(e, -127)).clamp(-127, 127)
    a = b.abs() / torch.exp2(e.double())[..., None]
    at = ((a > .25).int() + (a >= .75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5))
    return (at + 8 * torch.signbit(b)).view(x.shape), e


def values64(codes, e):
    v = GRID[(codes & 7).long()] * torch.where(codes >= 8, -1.0, 1.0)
    return v * torch.exp2(e.double()).repeat_interleave(32, 1)


def unpack(codes):
    c = codes.cpu().int()
    return torch.stack([c & 15, c >> 4], -1).view(c.shape[0], -1)


def scale_at(scales, R, K):
    """Scale bytes [R, K/32] from the tiled layout."""
    r, kb = torch.arange(R).view(-1, 1), torch.arange(K // 32).view(1, -1)
    kt = -(-K // 128)
    return scales.cpu()[((r // 128) * kt + kb // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + kb % 4].int()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("R,K", [(1, 32), (1, 4096), (3, 96), (77, 160), (128, 128), (129, 256), (300, 2048), (5, 8224)])
def test_quantize(R, K, dtype):
    g = torch.Generator().manual_seed(R + K)
    x = (torch.randn(R, K // 32, 32, generator=g) * torch.exp(8 * torch.randn(R, K // 32, 1, generator=g))).view(R, K)
    x = x.to(dtype)
    x.view(-1)[::7] = 0
    x.view(-1, 32)[0] = 0                                   # a block of zeros
    if R * K > 64:
        x.view(-1, 32)[1] = torch.linspace(-4, 4, 32).to(dtype)
    codes, scales = fp4_quantize(x.cuda())
    ec, ee = mx64(x)
    assert torch.equal(unpack(codes), ec)
    assert torch.equal(scale_at(scales, R, K), ee + 127)
    assert scales.numel() == -(-R // 128) * -(-K // 128) * 512
    full = scales.cpu().view(-1, -(-K // 128), 32, 4, 4)    # places past R or K hold 0
    pad = torch.zeros(-(-R // 128) * 128, -(-K // 128) * 4, dtype=torch.int32)
    pad[:R, :K // 32] = ee + 127
    got = full.permute(0, 3, 2, 1, 4).reshape(pad.shape)
    assert torch.equal(got.int(), pad)
    for dt in (torch.float32, torch.bfloat16):
        assert torch.equal(fp4_dequantize(codes, scales, dt).double().cpu(), values64(ec, ee))


def test_quantize_ties_extremes_and_non_finite():
    ties = torch.tensor([.25, .75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.9, 0.0])
    x = torch.zeros(6, 32)
    x[0, :10] = ties
    x[1, :10] = -ties
    x[2] = 3.3895e38                        # near the top of fp32
    x[3, 0], x[3, 1] = 1e-45, 3e-39         # subnormal
    x[4, 5] = float("inf")
    x[5, 5] = float("nan")
    codes, scales = fp4_quantize(x.cuda())
    ec, ee = mx64(x[:4])
    assert torch.equal(unpack(codes)[:4], ec)
    assert torch.equal(scale_at(scales, 6, 32)[:4], ee + 127)
    assert scale_at(scales, 6, 32)[4:].eq(255).all() and unpack(codes)[4:].eq(0).all()
    back = fp4_dequantize(codes, scales, torch.float32).cpu()
    assert torch.equal(back[:4].double(), values64(ec, ee)) and torch.isnan(back[4:]).all()


def routed(T, E, k, seed, hot=None):
    g = torch.Generator().manual_seed(seed)
    logits = torch.randn(T, E, generator=g)
    if hot is not None:
        logits[:, hot] += 100.0             # every token takes this expert
    return logits


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,d,E,k", [(1, 128, 4, 2), (37, 384, 8, 3), (500, 2048, 16, 8), (3, 256, 1, 1)])
def test_permute_fp4(T, d, E, k, dtype):
    x = torch.randn(T, d, generator=torch.Generator().manual_seed(T)).to(dtype)
    layer = MoELayerFp4(T, d, E, k, 256)
    L.moe_route_count_index(routed(T, E, k, 1).cuda(), k, layer.topk_idx, layer.topk_w, layer.counts, layer.offsets,
                            layer.tile_offsets, layer.row_of_slot, layer.token_of_row, layer.ws_index)
    layer.x_codes.fill_(0xEE)
    layer.x_scales.fill_(0xEE)
    L.moe_permute_fp4(x.cuda(), k, E, layer.row_of_slot, layer.counts, layer.tile_offsets, layer.x_codes, layer.x_scales)
    ec, ee = mx64(x)
    tor = layer.token_of_row.cpu().long()
    used = int(layer.tile_offsets[E]) * 128
    got, sc = unpack(layer.x_codes), scale_at(layer.x_scales, layer.rows_max, d)
    live = tor[:used] >= 0
    assert torch.equal(got[:used][live], ec[tor[:used][live]]) and torch.equal(sc[:used][live], (ee + 127)[tor[:used][live]])
    assert got[:used][~live].eq(0).all() and sc[:used][~live].eq(0).all()
    assert layer.x_codes[used:].eq(0xEE).all() and layer.x_scales[used // 128 * (d // 128) * 512:].eq(0xEE).all()


CASES = [  # T, d, E, k, f, hot
    (1, 256, 4, 2, 256, None), (1, 2048, 64, 8, 1024, None), (7, 512, 5, 1, 256, None), (129, 256, 3, 2, 512, 1),
    (300, 768, 8, 3, 256, None), (1500, 512, 2, 1, 512, 0), (2000, 1024, 37, 6, 768, None), (64, 2048, 8, 8, 1024, None),
]


@pytest.mark.parametrize("T,d,E,k,f,hot", CASES)
def test_grouped_ffn_fp4(T, d, E, k, f, hot):
    g = torch.Generator().manual_seed(T + d)
    x = torch.randn(T, d, generator=g).bfloat16().cuda()
    wgu = (torch.randn(E, 2 * f, d, generator=g) * 0.05).bfloat16().cuda()
    wd = (torch.randn(E, d, f, generator=g) * 0.05).bfloat16().cuda()
    W = Fp4Weights.quantize(wgu, wd)
    layer = MoELayerFp4(T, d, E, k, f)
    layer.y_perm.fill_(7.0)
    out = layer.forward(x, routed(T, E, k, T, hot).cuda(), W)
    assert layer.status() == (0, 0)
    xq = fp4_dequantize(*fp4_quantize(x)).double()
    gu, dn = fp4_dequantize(W.gate_up, W.gate_up_scales).double(), fp4_dequantize(W.down, W.down_scales).double()
    tor = layer.token_of_row.long()
    toff = layer.tile_offsets.cpu().tolist()
    counts = layer.counts.cpu().tolist()
    hv = fp4_dequantize(layer.h_codes, layer.h_scales, torch.float32).double()
    off = total = 0
    for e in range(E):
        r0, c = toff[e] * 128, counts[e]
        if c == 0:
            assert toff[e + 1] == toff[e]
            continue
        xe = xq[tor[r0:r0 + c]]
        ab = xe @ gu[e].T
        h = ab[:, :f] * torch.sigmoid(ab[:, :f]) * ab[:, f:]
        ec, ee = mx64(h)
        exp = values64(ec, ee).cuda()
        got = hv[r0:r0 + c]
        scale = torch.exp2(ee.double()).repeat_interleave(32, 1).cuda()
        assert ((got - exp).abs() <= 4 * scale).all()       # another code, or a scale across a power of two
        off += int((got != exp).sum())
        total += got.numel()
        ye = hv[r0:r0 + c] @ dn[e].T
        y = layer.y_perm[r0:r0 + c].double()
        top = ye.abs().max().item()
        assert ((y - ye).abs() <= 2.0 ** -8 * ye.abs() + 2e-5 * top).all()
        assert layer.y_perm[r0 + c:toff[e + 1] * 128].eq(0).all() and hv[r0 + c:toff[e + 1] * 128].eq(0).all()
    assert off <= max(2, 2e-3 * total), (off, total)
    assert layer.y_perm[toff[E] * 128:].eq(7.0).all()
    comb = (layer.y_perm[layer.row_of_slot.long()].double().view(T, k, d) * layer.topk_w.double()[..., None]).sum(1)
    assert ((out.double() - comb).abs() <= 2.0 ** -8 * comb.abs() + 1e-5 * comb.abs().max()).all()


def test_close_to_the_bf16_layer():
    """4-bit weights and tokens against the fp64 layer on the unquantised ones: E2M1 rounds with an error of about 0.1
    of the value, three times on the way, so the outputs agree in direction (cosine above 0.95)."""
    w = moe_inputs.small("fp4", T=96, d=512, E=8, k=2, f=512, dtype="bf16")
    inp = moe_inputs.make_all(w)
    layer = MoELayerFp4(w.T, w.d, w.E, w.k, w.f)
    out = layer.forward(inp["x"].cuda(), inp["logits"].cuda(), Fp4Weights.quantize(inp["w_gate_up"].cuda(), inp["w_down"].cuda()))
    idx, wt = oracle.route_topk(inp["logits"], w.k)
    assert torch.equal(layer.topk_idx.cpu(), idx)
    ref = oracle.moe_tokens(inp["x"], idx, wt, inp["w_gate_up"], inp["w_down"], inp["g"])["out"]
    assert torch.nn.functional.cosine_similarity(out.double().cpu().view(-1), ref.view(-1), dim=0).item() > 0.95


def test_repeats_bit_for_bit_on_another_stream_and_in_a_graph():
    T, d, E, k, f = 700, 512, 16, 4, 512
    g = torch.Generator().manual_seed(2)
    x = torch.randn(T, d, generator=g).bfloat16().cuda()
    W = Fp4Weights.quantize((torch.randn(E, 2 * f, d, generator=g) * 0.05).cuda(), (torch.randn(E, d, f, generator=g) * 0.05).cuda())
    logits = routed(T, E, k, 3).cuda()
    layer = MoELayerFp4(T, d, E, k, f)
    first = layer.forward(x, logits, W).clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    layer.forward(x, logits, W, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(layer.out, first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.forward(x, logits, W)
    layer.out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(layer.out, first) and layer.status() == (0, 0)


def test_non_finite_tokens_and_weights():
    """A token with a NaN or an infinity gives NaN rows of its own only; a weight, the features that it enters."""
    T, d, E, k, f = 40, 512, 4, 2, 256
    g = torch.Generator().manual_seed(9)
    x = torch.randn(T, d, generator=g).bfloat16()
    x[3, 100], x[17, 5] = float("nan"), float("inf")
    wgu = (torch.randn(E, 2 * f, d, generator=g) * 0.05).bfloat16()
    wd = (torch.randn(E, d, f, generator=g) * 0.05).bfloat16()
    layer = MoELayerFp4(T, d, E, k, f)
    logits = routed(T, E, k, 4).cuda()
    out = layer.forward(x.cuda(), logits, Fp4Weights.quantize(wgu.cuda(), wd.cuda())).float().cpu()
    bad = torch.zeros(T, dtype=torch.bool)
    bad[[3, 17]] = True
    assert torch.isnan(out[bad]).all() and torch.isfinite(out[~bad]).all()
    wd[1, 7, 3] = float("nan")                              # output feature 7 of expert 1
    x = torch.randn(T, d, generator=g).bfloat16().cuda()
    out = layer.forward(x, logits, Fp4Weights.quantize(wgu.cuda(), wd.cuda())).float().cpu()
    hit = (layer.topk_idx.cpu() == 1).any(1)
    assert torch.isnan(out[hit, 7]).all() and torch.isfinite(out[~hit]).all()
    rest = torch.ones(d, dtype=torch.bool)
    rest[7] = False
    assert torch.isfinite(out[:, rest]).all() and layer.status() == (0, 0)


def test_no_tokens():
    layer = MoELayerFp4(0, 256, 4, 2, 256)
    W = Fp4Weights.quantize(torch.randn(4, 512, 256, device="cuda"), torch.randn(4, 256, 256, device="cuda"))
    out = layer.forward(torch.empty((0, 256), dtype=torch.bfloat16, device="cuda"), torch.empty((0, 4), device="cuda"), W)
    assert out.shape == (0, 256) and layer.status() == (0, 0)


def test_refusals():
    x = torch.randn(4, 48, device="cuda")
    with pytest.raises(L.MoeError) as e:
        fp4_quantize(x)                                     # K is no multiple of 32
    assert e.value.code == -2
    x = torch.randn(8, 64, device="cuda")
    with pytest.raises(ValueError):
        fp4_quantize(x[:, ::2])
    with pytest.raises(TypeError):
        fp4_quantize(x.half())
    with pytest.raises(ValueError):
        L.moe_fp4_quantize(x, torch.empty((8, 32), dtype=torch.uint8, device="cuda"),
                           torch.empty(511, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        L.moe_fp4_quantize(x, torch.empty((8, 31), dtype=torch.uint8, device="cuda"),
                           torch.empty(512, dtype=torch.uint8, device="cuda"))
    layer = MoELayerFp4(4, 384, 2, 1, 256)                  # d is no multiple of 256
    W = Fp4Weights.quantize(torch.randn(2, 512, 384, device="cuda"), torch.randn(2, 384, 256, device="cuda"))
    with pytest.raises(L.MoeError) as e:
        layer.forward(torch.randn(4, 384, device="cuda").bfloat16(), torch.randn(4, 2, device="cuda"), W)
    assert e.value.code == -2
    W = Fp4Weights.quantize(torch.randn(3, 512, 256, device="cuda"), torch.randn(2, 256, 256, device="cuda"))
    with pytest.raises(ValueError):                         # weights of unlike expert counts
        MoELayerFp4(4, 256, 2, 1, 256).forward(torch.randn(4, 256, device="cuda").bfloat16(), torch.randn(4, 2, device="cuda"), W)


@pytest.mark.parametrize("T", [1, 96, 700])
def test_ffn_right_after_what_writes_its_inputs(T):
    """Offsets, weights and their scales written by the launches just before the call: the same result, bit for bit,
    as with them in place long before. (Both sets of kernels: few rows per expert, and many.)"""
    d, f, E, k = 512, 256, 4, 2
    g = torch.Generator().manual_seed(T)
    x = torch.randn(T, d, generator=g).to(torch.bfloat16).cuda()
    logits = torch.randn(T, E, generator=g).cuda()
    w = Fp4Weights.quantize((torch.randn(E, 2 * f, d, generator=g) * 0.05).cuda(), (torch.randn(E, d, f, generator=g) * 0.05).cuda())
    layer = MoELayerFp4(T, d, E, k, f)
    layer.y_perm.zero_()        # rows past the experts' are not written
    layer.forward(x, logits, w)
    want = layer.y_perm.clone()
    names = ("gate_up", "gate_up_scales", "down", "down_scales")
    kept = [getattr(w, n).clone() for n in names] + [layer.offsets.clone(), layer.tile_offsets.clone()]
    live = [getattr(w, n) for n in names] + [layer.offsets, layer.tile_offsets]
    args = (layer.x_codes, layer.x_scales, *live[:4], layer.tile_offsets, layer.offsets, layer.h_codes, layer.h_scales,
            layer.y_perm, layer.ws_ffn)
    for last in range(len(live)):
        for t in live:
            t.zero_()
        layer.y_perm.zero_()
        L.moe_permute_fp4(x, k, E, layer.row_of_slot, layer.counts, kept[5], layer.x_codes, layer.x_scales)
        for i in [j for j in range(len(live)) if j != last] + [last]:
            live[i].copy_(kept[i])
        L.moe_grouped_ffn_fwd_fp4(*args)
        assert torch.equal(layer.y_perm, want), last
    assert layer.status() == (0, 0)


@pytest.mark.parametrize("T,d,E,k,f,hot", [(3, 256, 256, 16, 256, None), (40, 256, 200, 2, 256, 150), (1, 256, 33, 1, 256, 32),
                                           (2600, 256, 70, 4, 256, 3), (9, 256, 256, 1, 256, 255)])
def test_many_experts_most_of_them_empty(T, d, E, k, f, hot):
    test_grouped_ffn_fp4(T, d, E, k, f, hot)


def test_few_tokens_in_buffers_for_many():
    """Buffers for 600 tokens per step, five used: the kernels are chosen by the buffers. Against buffers for five: at most
    2e-3 of h's codes fall on the other side of a rounding threshold (a step, at most half a value): with bf16
    outputs that is below 2e-2 of the output's norm."""
    T, d, E, k, f = 5, 512, 4, 2, 256
    g = torch.Generator().manual_seed(12)
    x = torch.randn(T, d, generator=g).bfloat16().cuda()
    W = Fp4Weights.quantize((torch.randn(E, 2 * f, d, generator=g) * 0.05).cuda(), (torch.randn(E, d, f, generator=g) * 0.05).cuda())
    logits = routed(T, E, k, 1).cuda()
    exp = MoELayerFp4(T, d, E, k, f).forward(x, logits, W).double()
    big = MoELayerFp4(600, d, E, k, f)
    idx, wt, slots = big.topk_idx[:T], big.topk_w[:T], big.row_of_slot[:T * k]
    L.moe_route_count_index(logits, k, idx, wt, big.counts, big.offsets, big.tile_offsets, slots, big.token_of_row, big.ws_index)
    L.moe_permute_fp4(x, k, E, slots, big.counts, big.tile_offsets, big.x_codes, big.x_scales)
    L.moe_grouped_ffn_fwd_fp4(big.x_codes, big.x_scales, W.gate_up, W.gate_up_scales, W.down, W.down_scales, big.tile_offsets,
                              big.offsets, big.h_codes, big.h_scales, big.y_perm, big.ws_ffn)
    out = torch.empty((T, d), dtype=torch.bfloat16, device="cuda")
    L.moe_combine_fwd(big.y_perm, wt, slots, T, k, out)
    assert big.status() == (0, 0)
    assert (out.double() - exp).norm() <= 2e-2 * exp.norm()
