"""Cases of the operators around one MoE layer: block norms, the AdamW step, and MXFP4 (4-bit microscaled) experts.

Each case runs one operator once. `run` has two forms: the plain one (elementary torch operations in 32 bits,
rounded once at the end) and, where `own` is true, the calls a user makes of the framework. `exact` gives the
operators' definitions in 64 bits.

Operators (the "op" of a case):
  norm      "part" pre or post, "dir" fwd or bwd: RMS norm before a block; after it, the norm of the block's
            output with its gate and the scaled residual, and the next block's norm in the same pass
  adamw     one AdamW step over many tensors, states in fp32 or in 8 bits (e4m3 codes, blocks of 256)
  quantize  MXFP4 quantisation (E2M1 codes, one E8M0 scale per 32 values) and reading it back
  experts   the layer's expert FFN on MXFP4 weights and tokens: tokens quantised into the grouped layout, both
            grouped products with SwiGLU and the quantisation of h between them, the weighted combine
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6
ADAM = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.1)
Q = 256            # values per scale of an 8-bit state
GROUP = 128        # rows to which each expert's rows are aligned in the grouped layout


def listed():
    return [
        # one decode step of a few sequences: latency of the fused norm, gate and residual
        dict(name="norm_post_fwd_decode", op="norm", part="post", dir="fwd", T=4, d=2048, dtype="bf16", gate="channel", next=True),
        # the training forward at the benchmark's token count
        dict(name="norm_post_fwd_train", op="norm", part="post", dir="fwd", T=8192, d=2048, dtype="bf16", gate="channel", next=True),
        # the training backward of the largest configuration
        dict(name="norm_post_bwd_large", op="norm", part="post", dir="bwd", T=16384, d=4096, dtype="bf16", gate="channel", next=True),
        # an fp32 model of odd width with a gate per token and channel
        dict(name="norm_post_bwd_f32_odd", op="norm", part="post", dir="bwd", T=1023, d=1537, dtype="f32", gate="token", next=True),
        # many small and odd tensors: launches and ragged ends
        dict(name="adamw_many_small", op="adamw", sizes="spread", count=300, largest=20011, dtype="f32", state="f32", master=False),
        # one layer's parameters with an fp32 master copy and fp32 states
        dict(name="adamw_layer_f32", op="adamw", sizes="layer", E=64, d=2048, f=1024, dtype="bf16", state="f32", master=True),
        # the same with 8-bit states and no master copy
        dict(name="adamw_layer_8bit", op="adamw", sizes="layer", E=64, d=2048, f=1024, dtype="bf16", state="f8", master=False),
        # an odd number of short fp32 rows
        dict(name="quantize_odd_f32", op="quantize", R=77, K=96, dtype="f32"),
        # a batch of tokens at the benchmark's size
        dict(name="quantize_tokens", op="quantize", R=16384, K=4096, dtype="bf16"),
        # decode: one token, its 8 experts' weights are the traffic
        dict(name="experts_decode", op="experts", T=1, d=2048, E=64, k=8, f=1024),
        # a small ragged batch: every expert has a few rows
        dict(name="experts_ragged", op="experts", T=333, d=2048, E=64, k=8, f=1024),
        # a prefill at the benchmark's token count
        dict(name="experts_prefill", op="experts", T=8192, d=2048, E=64, k=8, f=1024),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "adamw", "quantize", "experts", "experts"])
    if op == "norm":
        d = rng.choice([_spread(rng, 33, 4100), 64 * rng.randint(1, 64)])
        d = d + 8 if d == 3072 else d
        part = rng.choice(["pre", "post", "post"])
        return dict(op=op, part=part, dir=rng.choice(["fwd", "bwd"]), T=_spread(rng, 1, 16384), d=d,
                    dtype=rng.choice(["bf16", "f32"]) if d <= 2048 else "bf16",
                    gate=rng.choice(["none", "channel", "token"]) if part == "post" else "none",
                    next=part == "post" and rng.random() < 0.7)
    if op == "adamw":
        dtype = rng.choice(["bf16", "f32"])
        return dict(op=op, sizes="spread", count=rng.randint(1, 400), largest=_spread(rng, 100, 60_000_000), dtype=dtype,
                    state=rng.choice(["f32", "f8"]), master=dtype == "bf16" and rng.random() < 0.5)
    if op == "quantize":
        K = 32 * _spread(rng, 1, 128)
        K = K + 32 if K == 3072 else K
        return dict(op=op, R=_spread(rng, 1, 16384), K=K, dtype=rng.choice(["bf16", "f32"]) if K <= 2048 else "bf16")
    d, f, E = 256 * rng.randint(1, 8), 256 * rng.randint(1, 4), rng.choice([4, 8, 16, 37, 64])
    return dict(op=op, T=_spread(rng, 1, 8192), d=d, E=E, k=rng.randint(1, min(8, E)), f=f)


# ------------------------------------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def _sizes(c):
    if c["sizes"] == "layer":   # gate/up, down, router, the two norms' weights
        E, d, f = c["E"], c["d"], c["f"]
        return [E * 2 * f * d, E * d * f, E * d, d, d], [1.0, 1.0, 1.0, 0.0, 0.0]
    n, top = c["count"], c["largest"]
    sizes = [max(1, int(round(top ** ((i + 1) / n)))) for i in range(n)]
    return sizes, [0.0 if i % 3 == 0 else 1.0 for i in range(n)]


def _prepare_norm(c, g):
    T, d, dt = c["T"], c["d"], DTYPES[c["dtype"]]
    s = dict(case=c, x=_randn(g, (T, d), dt, 2.0), w=(1 + 0.2 * _randn(g, (d,), torch.float32)).to(dt))
    if c["part"] == "post":
        s["y"] = _randn(g, (T, d), dt, 0.5)
        s["gate"] = {"none": None, "channel": _randn(g, (d,), dt, 0.5), "token": _randn(g, (T, d), dt, 0.5)}[c["gate"]]
        s["w_next"] = (1 + 0.2 * _randn(g, (d,), torch.float32)).to(dt) if c["next"] else None
        s["scale"] = 0.75
    if c["dir"] == "bwd":
        s["dn"] = _randn(g, (T, d), dt) if c["part"] == "pre" or c["next"] else None
        s["dres"] = _randn(g, (T, d), dt)
        if c["part"] == "post":   # the stream after the block, as the forward stored it
            s["out"] = _randn(g, (T, d), dt, 1.7)
    if own:
        from mixture_experts_layer_histogram_gb300 import BlockNorms
        s["norms"] = BlockNorms(T, d, dt, gate=None if c["gate"] == "none" else c["gate"], res_scale=0.75, eps=EPS,
                                next_norm=c["next"])
    return s


def _prepare_adamw(c, g):
    sizes, decays = _sizes(c)
    blocks = [-(-n // Q) for n in sizes]
    starts = [0]
    for b in blocks:
        starts.append(starts[-1] + b)
    nb = starts[-1]
    dt = DTYPES[c["dtype"]]
    # one flat buffer per kind; every tensor starts at a multiple of 256 values
    live = torch.zeros(nb * Q, dtype=torch.bool, device="cuda")
    for n, b in zip(sizes, starts):
        live[b * Q:b * Q + n] = True
    def flat(scale):
        return torch.randn(nb * Q, generator=g, device="cuda").mul_(scale).mul_(live)
    s = dict(case=c, step=10)
    p = flat(0.02)
    s["p"] = p.to(dt)
    s["master"] = p if c["master"] else None
    s["g"] = flat(1e-3).to(dt)
    m, v = flat(3e-4), flat(1e-3).square_()
    if c["state"] == "f8":
        def hold(t):
            t = t.view(-1, Q)
            sc = t.abs().amax(1, keepdim=True) / 448.0
            return (t / sc.clamp_min(1e-30)).to(torch.float8_e4m3fn).view(-1), sc.view(-1).clone()
        s["m"], s["m_scale"] = hold(m)
        s["v"], s["v_scale"] = hold(v.sqrt_())
    else:
        s["m"], s["v"], s["m_scale"], s["v_scale"] = m, v, None, None
    # per 256-value block: the decay of its tensor and the place in it (tables that a step keeps)
    owner = torch.repeat_interleave(torch.arange(len(sizes), device="cuda"), torch.tensor(blocks, device="cuda"))
    s["wd"] = torch.tensor(decays, device="cuda")[owner] * ADAM["weight_decay"]
    s["place"] = (torch.arange(nb, device="cuda") - torch.tensor(starts[:-1], device="cuda")[owner]) * Q
    if own:
        from mixture_experts_layer_histogram_gb300 import AdamW
        def cut(t):
            return None if t is None else [t[b * Q:b * Q + n] for n, b in zip(sizes, starts)]
        def cut_scales(t):
            return None if t is None else [t[b:b + k] for k, b in zip(blocks, starts)]
        s["opt"] = AdamW(cut(s["p"]), cut(s["g"]), lr=ADAM["lr"], betas=(ADAM["beta1"], ADAM["beta2"]), eps=ADAM["eps"],
                         weight_decay=[ADAM["weight_decay"] * w for w in decays], state=c["state"],
                         masters=cut(s["master"]), m=cut(s["m"]), v=cut(s["v"]), m_scale=cut_scales(s["m_scale"]),
                         v_scale=cut_scales(s["v_scale"]), step=s["step"])
    return s


def _pack(x):
    """MXFP4 codes (two per byte, the even column low) and scales (the 128-row tile layout) of x [R, K]."""
    R, K = x.shape
    val, e = _mx_round(x)
    a = val.abs() * _exp2(-e).repeat_interleave(32, 1)
    code = ((a >= 0.5).int() + (a >= 1) + (a >= 1.5) + (a >= 2) + (a >= 3) + (a >= 4) + (a >= 6)) + 8 * (val < 0)
    codes = (code[:, 0::2] + 16 * code[:, 1::2]).to(torch.uint8)
    RT, KT = -(-R // 128), -(-K // 128)
    sc = torch.zeros(RT * 128, KT * 4, dtype=torch.uint8, device=x.device)
    sc[:R, :K // 32] = (e + 127).to(torch.uint8)
    return codes, sc.view(RT, 4, 32, KT, 4).permute(0, 3, 2, 1, 4).reshape(-1).contiguous()


def _prepare_experts(c, g):
    T, d, E, k, f = (c[n] for n in ("T", "d", "E", "k", "f"))
    s = dict(case=c, x=_randn(g, (T, d), torch.bfloat16))
    logits = torch.randn(T, E, generator=g, device="cuda")
    w, idx = logits.topk(k, 1)
    s["topk_w"] = torch.softmax(w, 1)
    idx = idx.reshape(-1)
    counts = torch.bincount(idx, minlength=E)
    tiles = torch.zeros(E + 1, dtype=torch.int64, device="cuda")
    tiles[1:] = torch.cumsum((counts + GROUP - 1) // GROUP, 0)
    offs = torch.zeros(E + 1, dtype=torch.int64, device="cuda")
    offs[1:] = torch.cumsum(counts, 0)
    order = torch.argsort(idx, stable=True)
    rank = torch.empty_like(order)
    rank[order] = torch.arange(T * k, device="cuda")
    rank = rank - offs[idx]
    s["row_of_slot"] = (tiles[idx] * GROUP + rank).int()
    s["counts"], s["offsets"], s["tile_offsets"] = counts.int(), offs.int(), tiles.int()
    s["experts"] = counts.nonzero().view(-1)                       # the experts that have rows
    s["cap"] = int(counts.max())
    at = torch.zeros(E, dtype=torch.int64, device="cuda")
    at[s["experts"]] = torch.arange(len(s["experts"]), device="cuda")
    s["slot"] = at[idx] * s["cap"] + rank
    s["rows_max"] = -(-(T * k + E * (GROUP - 1)) // GROUP) * GROUP
    parts = [_pack(_randn(g, (2 * f, d), torch.bfloat16, 0.02)) for _ in range(E)]
    s["wgu"], s["wgu_s"] = torch.stack([p[0] for p in parts]), torch.cat([p[1] for p in parts])
    parts = [_pack(_randn(g, (d, f), torch.bfloat16, 0.02)) for _ in range(E)]
    s["wd"], s["wd_s"] = torch.stack([p[0] for p in parts]), torch.cat([p[1] for p in parts])
    if own:
        from mixture_experts_layer_histogram_gb300 import _lib as L
        R = s["rows_max"]
        u8 = dict(dtype=torch.uint8, device="cuda")
        s["xq"], s["xq_s"] = torch.empty((R, d // 2), **u8), torch.empty(L.moe_fp4_scale_bytes(R, d), **u8)
        s["hq"], s["hq_s"] = torch.empty((R, f // 2), **u8), torch.empty(L.moe_fp4_scale_bytes(R, f), **u8)
        s["y"] = torch.empty((R, d), dtype=torch.bfloat16, device="cuda")
        s["out"] = torch.empty((T, d), dtype=torch.bfloat16, device="cuda")
        s["ws"] = torch.zeros(L.moe_grouped_ffn_workspace_size(E, d, f, R, L.MOE_BF16, False), **u8)
    return s


def prepare(case, seed):
    g = _gen(seed)
    if case["op"] == "norm":
        return _prepare_norm(case, g)
    if case["op"] == "adamw":
        return _prepare_adamw(case, g)
    if case["op"] == "experts":
        return _prepare_experts(case, g)
    R, K, dt = case["R"], case["K"], DTYPES[case["dtype"]]
    spread = torch.exp(torch.randn(R, K // 32, 1, generator=g, device="cuda") * 2)   # blocks of unlike magnitude
    x = (torch.randn(R, K // 32, 32, generator=g, device="cuda") * spread).view(R, K).to(dt)
    s = dict(case=case, x=x)
    if own:
        from mixture_experts_layer_histogram_gb300 import _lib as L
        s["codes"] = torch.empty((R, K // 2), dtype=torch.uint8, device="cuda")
        s["scales"] = torch.empty(L.moe_fp4_scale_bytes(R, K), dtype=torch.uint8, device="cuda")
        s["values"] = torch.empty_like(x)
    return s


# ------------------------------------------------------------------------------------------------ plain forms
def _rms(v):
    return torch.rsqrt((v * v).mean(1, keepdim=True) + EPS)


def _norm_back(dn, x, w):
    """Gradients of n = x rms(x) w with respect to x and w."""
    r, u = _rms(x), dn * w
    return r * (u - x * (r * r * (u * x).mean(1, keepdim=True))), (dn * x * r).sum(0)


def _plain_norm(s):
    c = s["case"]
    dt = DTYPES[c["dtype"]]
    f = {n: t.float() for n, t in s.items() if isinstance(t, torch.Tensor)}
    if c["part"] == "pre":
        if c["dir"] == "fwd":
            return {"n": (f["x"] * _rms(f["x"]) * f["w"]).to(dt)}
        dx, dw = _norm_back(f["dn"], f["x"], f["w"])
        return {"dx": (dx + f["dres"]).to(dt), "dw": dw.to(dt)}
    gate = f.get("gate", torch.ones((), device="cuda"))
    if c["dir"] == "fwd":
        out = s["scale"] * f["x"] + gate * (f["y"] * _rms(f["y"]) * f["w"])
        res = {"out": out.to(dt)}
        if c["next"]:
            res["n"] = (out * _rms(out) * f["w_next"]).to(dt)
        return res
    G, res = f["dres"], {}
    if c["next"]:
        dG, dwn = _norm_back(f["dn"], f["out"], f["w_next"])
        G = G + dG
        res["dw_next"] = dwn.to(dt)
    dy, dw = _norm_back(G * gate, f["y"], f["w"])
    res.update(dx=(s["scale"] * G).to(dt), dy=dy.to(dt), dw_post=dw.to(dt))
    if c["gate"] != "none":
        dg = G * f["y"] * _rms(f["y"]) * f["w"]
        res["d_gate"] = (dg.sum(0) if c["gate"] == "channel" else dg).to(dt)
    return res


# Dither of values that are kept in few bits only: a Weyl sequence over the place in the tensor and the step
DITHER_I, DITHER_T = 2654435769, 1640531535


def _dither(s, step, shift):
    i = s["place"][:, None] + torch.arange(Q, device="cuda")
    return ((i * DITHER_I + step * DITHER_T + shift) & 0xFFFFFFFF) >> 12     # 20 bits


def _bits(v):
    return v.view(torch.int32)


def _dithered_e4m3(y, u):
    """y (|y| <= 448, fp32) to e4m3: down to the grid of y's binade after adding u/2^20 of its step."""
    a = y.abs()
    normal = (_bits(a) + u.int()) & -(1 << 20)
    small = ((a * 536870912.0).int() + u.int()) >> 20                        # steps of 2^-9 below 2^-6
    a = torch.where(a < 0.015625, small.float() * 0.001953125, normal.view(torch.float32)).clamp_max(448.0)
    return torch.where(y < 0, -a, a).to(torch.float8_e4m3fn)


def _plain_adamw(s):
    c, a = s["case"], ADAM
    s["step"] += 1
    t = s["step"]
    b1, b2 = 1 - a["beta1"] ** t, 1 - a["beta2"] ** t
    g = s["g"].float().view(-1, Q)
    m, v = s["m"].float().view(-1, Q), s["v"].float().view(-1, Q)
    if c["state"] == "f8":
        m, v = m * s["m_scale"][:, None], (v * s["v_scale"][:, None]).square()
    m = a["beta1"] * m + (1 - a["beta1"]) * g
    v = a["beta2"] * v + (1 - a["beta2"]) * (g * g)
    root = v.sqrt()
    p = (s["master"] if c["master"] else s["p"]).float().view(-1, Q)
    p = p * (1 - a["lr"] * s["wd"])[:, None] - (a["lr"] / b1) * m / (root / math.sqrt(b2) + a["eps"])
    res = {}
    if c["state"] == "f8":
        for name, val, shift in (("m", m, 0), ("v", root, 0x55555555)):
            top = val.abs().amax(1, keepdim=True)
            keep = top >= 1e-30
            y = val * torch.where(keep, 448.0 / top, 0.0)
            s[name].copy_(_dithered_e4m3(y, _dither(s, t, shift)).view(-1))
            s[name + "_scale"].copy_(torch.where(keep, top / 448.0, 0.0).view(-1))
            res[name + "_scale"] = s[name + "_scale"]
    else:
        s["m"].copy_(m.view(-1))
        s["v"].copy_(v.view(-1))
    if c["master"]:
        s["master"].copy_(p.view(-1))
        res["master"] = s["master"]
    elif c["dtype"] == "bf16":
        p = ((_bits(p) + (_dither(s, t, 0xAAAAAAAA) >> 4).int()) & -65536).view(torch.float32)
    s["p"].copy_(p.view(-1))
    return dict(res, p=s["p"], m=s["m"], v=s["v"])


def _exp2(e):
    """2^e as fp32 for integers -126 <= e <= 127."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _mx_round(x):
    """The values that MXFP4 holds for x [R, K] (fp32), and the exponents of the scales [R, K/32]."""
    b = x.float().view(x.shape[0], -1, 32)
    e = (torch.frexp(b.abs().amax(2, keepdim=True))[1] - 3).clamp(-127, 127)
    y = (b * _exp2(-e)).clamp(-6, 6)
    a = y.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    v = torch.round(y / step) * step
    half = e >> 1                                                            # 2^e in two factors: e may be -127
    return (v * _exp2(half) * _exp2(e - half)).view(x.shape), e.squeeze(2)


def _unpack(codes, scales):
    """[n, R, K/2] codes and [n, tiles] scales (R and K multiples of 128) to fp32 values [n, R, K]."""
    n, R, K = codes.shape[0], codes.shape[1], codes.shape[2] * 2
    lut = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6], device=codes.device)
    v = lut[torch.stack([codes & 15, codes >> 4], 3).view(n, R, K).int()]
    sc = scales.view(n, R // 128, K // 128, 32, 4, 4).permute(0, 1, 4, 3, 2, 5).reshape(n, R, K // 32)
    return v.view(n, R, K // 32, 32).mul_(_exp2(sc.int() - 127)[..., None]).view(n, R, K)


def _plain_experts(s):
    c = s["case"]
    T, d, E, k, f = (c[n] for n in ("T", "d", "E", "k", "f"))
    on = s["experts"]
    xq = _mx_round(s["x"])[0]
    xg = torch.zeros(len(on) * s["cap"], d, device="cuda")
    xg[s["slot"]] = xq.repeat_interleave(k, 0)
    ab = torch.bmm(xg.view(len(on), -1, d), _unpack(s["wgu"][on], s["wgu_s"].view(E, -1)[on]).transpose(1, 2))
    a, b = ab[..., :f], ab[..., f:]
    h = a / (1 + torch.exp(-a)) * b
    hq = _mx_round(h.reshape(-1, f))[0].view(len(on), -1, f)
    y = torch.bmm(hq, _unpack(s["wd"][on], s["wd_s"].view(E, -1)[on]).transpose(1, 2)).view(-1, d)
    return {"out": (y[s["slot"]].view(T, k, d) * s["topk_w"][..., None]).sum(1).to(torch.bfloat16)}


# ------------------------------------------------------------------------------------------------ one pass
def _own(s):
    c = s["case"]
    if c["op"] == "norm":
        nm = s["norms"]
        if c["part"] == "pre":
            return {"n": nm.pre(s["x"], s["w"])} if c["dir"] == "fwd" else nm.pre_backward(s["dn"], s["x"], s["w"], dx_in=s["dres"])
        if c["dir"] == "bwd":
            return nm.post_backward(s["dres"], s["dn"], s["out"], s["y"], s["w"], gate=s["gate"], w_next=s["w_next"])
        out, n = nm.post(s["y"], s["x"], s["w"], gate=s["gate"], w_next=s["w_next"])
        return {"out": out, "n": n} if c["next"] else {"out": out}
    if c["op"] == "adamw":
        s["opt"].step()
        res = dict(p=s["p"], m=s["m"], v=s["v"])
        if c["state"] == "f8":
            res.update(m_scale=s["m_scale"], v_scale=s["v_scale"])
        if c["master"]:
            res["master"] = s["master"]
        return res
    from mixture_experts_layer_histogram_gb300 import _lib as L
    if c["op"] == "quantize":
        L.moe_fp4_quantize(s["x"], s["codes"], s["scales"])
        L.moe_fp4_dequantize(s["codes"], s["scales"], s["values"])
        return {"values": s["values"]}
    L.moe_permute_fp4(s["x"], c["k"], c["E"], s["row_of_slot"], s["counts"], s["tile_offsets"], s["xq"], s["xq_s"])
    L.moe_grouped_ffn_fwd_fp4(s["xq"], s["xq_s"], s["wgu"], s["wgu_s"], s["wd"], s["wd_s"], s["tile_offsets"],
                              s["offsets"], s["hq"], s["hq_s"], s["y"], s["ws"])
    L.moe_combine_fwd(s["y"], s["topk_w"], s["row_of_slot"], c["T"], c["k"], s["out"])
    return {"out": s["out"]}


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "norm":
        return _plain_norm(state)
    if op == "adamw":
        return _plain_adamw(state)
    if op == "quantize":
        return {"values": _mx_round(state["x"])[0].to(state["x"].dtype)}
    return _plain_experts(state)


def work(case):
    c = case
    if c["op"] == "norm":
        T, d, z = c["T"], c["d"], 2 if c["dtype"] == "bf16" else 4
        token = c["part"] == "post" and c["gate"] == "token"
        channel = c["part"] == "post" and c["gate"] == "channel"
        if c["part"] == "pre":
            rows, vecs = (2, 1) if c["dir"] == "fwd" else (4, 2)
        elif c["dir"] == "fwd":
            rows, vecs = 3 + c["next"] + token, 1 + c["next"] + channel
        else:
            rows, vecs = 4 + 2 * c["next"] + 2 * token, 2 + 2 * c["next"] + 2 * channel
        return {"bytes": (rows * T * d + vecs * d) * z, "flops": 8 * rows * T * d}
    if c["op"] == "adamw":
        n = sum(_sizes(c)[0])
        z = 2 if c["dtype"] == "bf16" else 4
        per = z + z + (8 if c["master"] else z)          # gradient; parameter written; master read and written, or parameter read
        per += 16 if c["state"] == "f32" else 4 + 16 / Q
        return {"bytes": per * n, "flops": 15 * n}
    if c["op"] == "quantize":
        n, z = c["R"] * c["K"], 2 if c["dtype"] == "bf16" else 4
        return {"bytes": n * (2 * z + 17 / 32), "flops": 5 * n}
    T, d, E, k, f = (c[n] for n in ("T", "d", "E", "k", "f"))
    on = E * (1 - (1 - k / E) ** T)                       # experts with rows, on average
    return {"bytes": on * 3 * d * f * 17 / 32 + 4 * T * d + 8 * T * k, "flops": 6 * T * k * d * f}


# ------------------------------------------------------------------------------------------------ in 64 bits
def _exact_norm(s):
    c = s["case"]
    D = {n: t.double() for n, t in s.items() if isinstance(t, torch.Tensor)}

    def grads(dn, x, w):
        var = x.pow(2).sum(1, keepdim=True) / x.shape[1] + EPS
        r = var.pow(-0.5)
        dot = (dn * w * x).sum(1, keepdim=True) / x.shape[1]
        return dn * w * r - x * dot * var.pow(-1.5), torch.einsum("td,td->d", dn, x * r)

    def norm(x, w):
        return x / torch.sqrt(x.pow(2).sum(1, keepdim=True) / x.shape[1] + EPS) * w

    if c["part"] == "pre":
        if c["dir"] == "fwd":
            return {"n": norm(D["x"], D["w"])}
        dx, dw = grads(D["dn"], D["x"], D["w"])
        return {"dx": D["dres"] + dx, "dw": dw}
    gate = D["gate"] if s["gate"] is not None else torch.ones(1, dtype=torch.float64, device="cuda")
    if c["dir"] == "fwd":
        out = D["x"] * s["scale"] + gate * norm(D["y"], D["w"])
        return {"out": out, "n": norm(out, D["w_next"])} if c["next"] else {"out": out}
    res, G = {}, D["dres"]
    if c["next"]:
        more, res["dw_next"] = grads(D["dn"], D["out"], D["w_next"])
        G = G + more
    res["dx"] = G * s["scale"]
    res["dy"], res["dw_post"] = grads(G * gate, D["y"], D["w"])
    if c["gate"] != "none":
        res["d_gate"] = G * norm(D["y"], D["w"])
        if c["gate"] == "channel":
            res["d_gate"] = res["d_gate"].sum(0)
    return res


def _exact_adamw(s):
    c, a, t = s["case"], ADAM, s["step"] + 1

    def weyl(shift):
        i = (s["place"].view(-1, 1) + torch.arange(Q, device="cuda").view(1, -1)) % (1 << 32)
        return torch.div((i * DITHER_I + (t * DITHER_T + shift)) % (1 << 32), 4096, rounding_mode="floor")

    g = s["g"].double().view(-1, Q)
    m, r = s["m"].double().view(-1, Q), s["v"].double().view(-1, Q)
    if c["state"] == "f8":
        m, v = m * s["m_scale"].double().view(-1, 1), (r * s["v_scale"].double().view(-1, 1)) ** 2
    else:
        v = r
    m = m + (1 - a["beta1"]) * (g - m)
    v = v + (1 - a["beta2"]) * (g ** 2 - v)
    p = (s["master"] if c["master"] else s["p"]).double().view(-1, Q)
    p = p - a["lr"] * s["wd"].double().view(-1, 1) * p
    p = p - a["lr"] * (m / (1 - a["beta1"] ** t)) / ((v / (1 - a["beta2"] ** t)) ** 0.5 + a["eps"])
    res = {}
    if c["state"] == "f8":
        for name, val, shift in (("m", m, 0), ("v", v ** 0.5, 0x55555555)):
            scale = val.abs().max(1, keepdim=True).values / 448
            y = torch.where(scale > 0, val / scale, torch.zeros_like(val)).abs()
            ulp = torch.exp2(torch.floor(torch.log2(y.clamp_min(2.0 ** -6))) - 3)
            y = (torch.floor(y / ulp + weyl(shift) / 2.0 ** 20) * ulp).clamp_max(448)
            res[name] = (torch.sign(val) * y).view(-1)
            res[name + "_scale"] = scale.view(-1)
    else:
        res = {"m": m.view(-1), "v": v.view(-1)}
    if c["master"]:
        res["master"] = p.view(-1)
    elif c["dtype"] == "bf16":
        q = p.abs().clamp_min(2.0 ** -126)
        ulp = torch.exp2(torch.floor(torch.log2(q)) - 7)
        p = torch.sign(p) * torch.floor(p.abs() / ulp + (weyl(0xAAAAAAAA) // 16) / 2.0 ** 16) * ulp
    res["p"] = p.view(-1)
    return res


def _exact_quantize(x):
    """MXFP4 values of x [R, K] in 64 bits: each magnitude against the midpoints of the seven steps of E2M1."""
    b = x.double().view(x.shape[0], -1, 32)
    top = b.abs().max(2, keepdim=True).values
    e = torch.floor(torch.log2(top.clamp_min(2.0 ** -149)))
    e = e - (torch.exp2(e) > top).double() + (torch.exp2(e + 1) <= top).double()   # the logarithm may round across
    scale = torch.exp2((e - 2).clamp(-127, 127))
    a = (b / scale).abs()
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=x.device)
    at = (a > 0.25).long() + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5)
    return (torch.sign(b) * grid[at] * scale).view(x.shape)


def _exact_experts(s):
    c = s["case"]
    T, d, E, k, f = (c[n] for n in ("T", "d", "E", "k", "f"))
    grid = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64, device="cuda")

    def values(codes, scales):
        R, K = codes.shape[0], codes.shape[1] * 2
        v = torch.empty(R, K, dtype=torch.float64, device="cuda")
        v[:, 0::2], v[:, 1::2] = grid[(codes % 16).long()], grid[(codes // 16).long()]
        r, q = torch.arange(R, device="cuda").view(-1, 1), torch.arange(K // 32, device="cuda").view(1, -1)
        place = ((r // 128) * (K // 128) + q // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + q % 4
        return v * torch.exp2(scales[place].double() - 127).repeat_interleave(32, 1)

    x = _exact_quantize(s["x"])
    weight = s["topk_w"].double().reshape(-1)
    row = s["row_of_slot"].long()
    first = s["tile_offsets"].long() * GROUP
    out = torch.zeros(T, d, dtype=torch.float64, device="cuda")
    for e in s["experts"].tolist():
        slots = ((row >= first[e]) & (row < first[e + 1])).nonzero().view(-1)
        tok = slots // k
        ab = x[tok] @ values(s["wgu"][e], s["wgu_s"].view(E, -1)[e]).T
        h = ab[:, :f] * torch.sigmoid(ab[:, :f]) * ab[:, f:]
        y = _exact_quantize(h) @ values(s["wd"][e], s["wd_s"].view(E, -1)[e]).T
        out.index_add_(0, tok, y * weight[slots].view(-1, 1))
    return {"out": out}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        return _exact_norm(s)
    if case["op"] == "adamw":
        return _exact_adamw(s)
    if case["op"] == "quantize":
        return {"values": _exact_quantize(s["x"])}
    return _exact_experts(s)
