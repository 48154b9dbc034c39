"""Cases of a block's further operators: layer norm, the gated feed-forward block, and activation checkpoints in 8 bits.

Each case runs its operators once. `run` has two forms: the plain one (elementary torch operations in 32 bits,
rounded once at the end) and, where `own` is true, the calls a user makes of the framework. `exact` gives the
operators' definitions in 64 bits.

Operators (the "op" of a case):
  layernorm  "dir" fwd or bwd: x to (x - mean) / sqrt(var + eps) * w + b, and its gradients (dx added to the one that
             reaches x past the norm); "dir" kept: the forward keeps its normalised rows in 8 bits, and the backward
             restores the norm's output and forms the gradients from those
  ffn        h = act(x Wg^T) * (x Wu^T), y = h Wd^T (added to `add` where there is one): "dir" fwd, or step: the
             forward and the backward pass; "keep" f8: the gate and up projections are kept in 8 bits between them
  act8       a tensor to 8 bits (e4m3 codes, one power of two per 32 values of a row) and back
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-5
GELU_C, GELU_K = math.sqrt(2 / math.pi), 0.044715


def listed():
    return [
        # one decode step of a few sequences: latency
        dict(name="layernorm_fwd_decode", op="layernorm", dir="fwd", T=4, d=2048, dtype="bf16", bias=True),
        # the training backward at the widest configuration
        dict(name="layernorm_bwd_large", op="layernorm", dir="bwd", T=16384, d=4096, dtype="bf16", bias=True),
        # an fp32 model of odd width
        dict(name="layernorm_bwd_f32_odd", op="layernorm", dir="bwd", T=1023, d=1537, dtype="f32", bias=True),
        # a training step's norm at the benchmark's token count that keeps 8 bits per value for its backward
        dict(name="layernorm_kept_train", op="layernorm", dir="kept", T=8192, d=2048, dtype="bf16", bias=True),
        # one token through the expert that every token takes, added to the routed experts' output
        dict(name="ffn_fwd_one_token", op="ffn", dir="fwd", T=1, d=2048, f=1024, dtype="bf16", act="silu", keep="none", add=True),
        # a decode batch through a wide dense block: the weights are the traffic
        dict(name="ffn_fwd_decode_batch", op="ffn", dir="fwd", T=24, d=4096, f=8192, dtype="bf16", act="gelu", keep="none", add=False),
        # a short ragged prompt
        dict(name="ffn_fwd_prompt_ragged", op="ffn", dir="fwd", T=777, d=2048, f=1024, dtype="bf16", act="silu", keep="none", add=True),
        # a training step of that expert at the benchmark's token count
        dict(name="ffn_step_train", op="ffn", dir="step", T=8192, d=2048, f=1024, dtype="bf16", act="silu", keep="all", add=True),
        # a training step of a wide dense block that keeps its projections in 8 bits
        dict(name="ffn_step_kept_large", op="ffn", dir="step", T=8192, d=4096, f=8192, dtype="bf16", act="silu", keep="f8", add=False),
        # an fp32 model of odd sizes
        dict(name="ffn_step_f32_odd", op="ffn", dir="step", T=203, d=501, f=1337, dtype="f32", act="gelu", keep="all", add=False),
        # a few odd fp32 rows
        dict(name="act8_odd_f32", op="act8", R=77, K=999, dtype="f32"),
        # a layer's saved activations
        dict(name="act8_tokens", op="act8", R=16384, K=4096, dtype="bf16"),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["layernorm", "layernorm", "ffn", "ffn", "ffn", "act8"])
    if op == "layernorm":
        d = rng.choice([_spread(rng, 33, 8192), 64 * rng.randint(1, 96)])
        kind = rng.choice(["fwd", "bwd", "kept"])
        return dict(op=op, dir=kind, T=_spread(rng, 1, 16384), d=d, dtype="bf16" if kind == "kept" or d > 2048 else rng.choice(["bf16", "f32"]),
                    bias=rng.random() < 0.7)
    if op == "act8":
        return dict(op=op, R=_spread(rng, 1, 16384), K=_spread(rng, 1, 4100), dtype=rng.choice(["bf16", "f32"]))
    kind, act, add = rng.choice(["fwd", "fwd", "step"]), rng.choice(["silu", "gelu"]), rng.random() < 0.5
    if rng.random() < 0.2:
        return dict(op=op, dir=kind, T=_spread(rng, 1, 700), d=_spread(rng, 16, 1400), f=_spread(rng, 16, 1400), dtype="f32", act=act,
                    keep="none" if kind == "fwd" else "all", add=add)
    keep = "none" if kind == "fwd" else rng.choice(["all", "f8"])
    unit = 32 if keep == "f8" else 8
    return dict(op=op, dir=kind, T=_spread(rng, 1, 8192), d=8 * _spread(rng, 8, 512), f=unit * _spread(rng, 2, 8192 // unit), dtype="bf16", act=act,
                keep=keep, add=add)


# ------------------------------------------------------------------------------------------------ inputs
def _randn(g, shape, dtype, scale=1.0, shift=0.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale + shift).to(dtype)


def prepare(case, seed):
    c, g = case, torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[c["dtype"]]
    s = dict(case=c)
    if c["op"] == "act8":
        R, K = c["R"], c["K"]
        spread = torch.exp(torch.randn(R, -(-K // 32), generator=g, device="cuda") * 2).repeat_interleave(32, 1)[:, :K]   # blocks of unlike magnitude
        s["x"] = (torch.randn(R, K, generator=g, device="cuda") * spread).to(dt)
        if own:
            from mixture_experts_layer_histogram_gb300 import _lib as L
            s["codes"] = torch.empty((R, K), dtype=torch.uint8, device="cuda")
            s["scales"] = torch.empty(L.moe_act8_scale_bytes(R, K), dtype=torch.uint8, device="cuda")
            s["values"] = torch.empty_like(s["x"])
        return s
    T, d = c["T"], c["d"]
    if c["op"] == "layernorm":
        rows = torch.exp(0.5 * torch.randn((T, 1), generator=g, device="cuda"))          # rows of unlike scale, not centred
        s["x"] = (rows * torch.randn((T, d), generator=g, device="cuda") + 0.5).to(dt)
        s["w"], s["b"] = _randn(g, (d,), dt, 0.2, 1.0), _randn(g, (d,), dt, 0.2) if c["bias"] else None
        if c["dir"] != "fwd":
            s["dn"], s["dres"] = _randn(g, (T, d), dt), _randn(g, (T, d), dt)
        if own:
            from mixture_experts_layer_histogram_gb300 import LayerNorm
            s["norm"] = LayerNorm(T, d, dt, eps=EPS, bias=c["bias"], keep="f8" if c["dir"] == "kept" else None, backward=c["dir"] != "fwd")
            if c["dir"] == "kept":
                s["again"] = torch.empty((T, d), dtype=dt, device="cuda")
        if c["dir"] == "bwd":   # what the forward left for the backward
            x = s["x"].double()
            m = x.mean(1)
            s["mean"], s["rstd"] = m.float(), ((x - m[:, None]).square().mean(1) + EPS).rsqrt().float()
            if own:
                s["norm"].mean.copy_(s["mean"])
                s["norm"].rstd.copy_(s["rstd"])
        return s
    f = c["f"]
    s["x"] = _randn(g, (T, d), dt)
    s["wgu"], s["wd"] = _randn(g, (2 * f, d), dt, d ** -0.5), _randn(g, (d, f), dt, f ** -0.5)
    s["add"] = _randn(g, (T, d), dt) if c["add"] else None
    if c["dir"] == "step":
        s["dy"] = _randn(g, (T, d), dt)
        s["dadd"] = _randn(g, (T, d), dt) if c["add"] else None     # the gradient that reaches x past the block
    if own:
        from mixture_experts_layer_histogram_gb300 import GatedFFN
        s["ffn"] = GatedFFN(T, d, f, dt, act=c["act"], keep="f8" if c["keep"] == "f8" else None, backward=c["dir"] == "step")
    return s


# ------------------------------------------------------------------------------------------------ plain forms
def _exp2(e):
    """2^e as fp32 for integers -126 <= e <= 127."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _round8(x):
    """The values that 8 bits hold for x [R, K] (fp32): e4m3 codes of x / 2^e, 2^e the least power of two with max |x| <= 448 2^e in a block of 32."""
    R, K = x.shape
    b = torch.nn.functional.pad(x, (0, -K % 32)).view(R, -1, 32)
    m, e = torch.frexp(b.abs().amax(2, keepdim=True))                     # max = m 2^e, 0.5 <= m < 1; 448 = 0.875 2^9
    e = (e - 9 + (m > 0.875).int()).clamp_min(-127)
    half = -e >> 1                                                        # 2^-e in two factors: -e may be 127 and more
    y = b * _exp2(half) * _exp2(-e - half)
    step = _exp2(torch.frexp(y.abs().clamp_min(2.0 ** -6))[1] - 4)        # 2^-3 of the binade, 2^-9 below 2^-6
    v = torch.round(y / step) * step
    half = e >> 1
    return (v * _exp2(half) * _exp2(e - half)).view(R, -1)[:, :K]


def _plain_layernorm(s):
    c, dt = s["case"], DTYPES[s["case"]["dtype"]]
    x, w = s["x"].float(), s["w"].float()
    b = s["b"].float() if c["bias"] else torch.zeros((), device="cuda")
    if c["dir"] == "bwd":
        m, r = s["mean"][:, None], s["rstd"][:, None]
    else:
        m = x.mean(1, keepdim=True)
        r = torch.rsqrt((x - m).square().mean(1, keepdim=True) + EPS)
    xh, res = (x - m) * r, {}
    if c["dir"] != "bwd":
        res["n"] = (xh * w + b).to(dt)
        if c["dir"] == "fwd":
            return res
        xh = _round8(xh)
        res["again"] = (xh * w + b).to(dt)
    dn = s["dn"].float()
    u = dn * w
    dx = r * (u - u.mean(1, keepdim=True) - xh * (u * xh).mean(1, keepdim=True)) + s["dres"].float()
    res.update(dx=dx.to(dt), dw=(dn * xh).sum(0).to(dt))
    if c["bias"]:
        res["db"] = dn.sum(0).to(dt)
    return res


def _plain_gate(a, kind):
    """act(a) and its derivative."""
    if kind == "silu":
        p = 1 / (1 + torch.exp(-a))
        return a * p, p * (1 + a * (1 - p))
    t = torch.tanh(GELU_C * (a + GELU_K * a * a * a))
    return 0.5 * a * (1 + t), 0.5 * (1 + t) + 0.5 * a * (1 - t * t) * GELU_C * (1 + 3 * GELU_K * a * a)


def _plain_ffn(s):
    c, dt, f = s["case"], DTYPES[s["case"]["dtype"]], s["case"]["f"]
    x, wgu, wd = s["x"].float(), s["wgu"].float(), s["wd"].float()
    ab = x @ wgu.T
    h = _plain_gate(ab[:, :f], c["act"])[0] * ab[:, f:]
    y = h @ wd.T
    res = {"y": (y + s["add"].float() if c["add"] else y).to(dt)}
    if c["dir"] == "fwd":
        return res
    if c["keep"] == "f8":
        ab = _round8(ab)
    a, b, dy = ab[:, :f], ab[:, f:], s["dy"].float()
    g, dg = _plain_gate(a, c["act"])
    dh = dy @ wd
    dab = torch.cat([dh * b * dg, dh * g], 1)
    dx = dab @ wgu
    res.update(dx=(dx + s["dadd"].float() if c["add"] else dx).to(dt), dw_gate_up=(dab.T @ x).to(dt), dw_down=(dy.T @ (g * b)).to(dt))
    return res


# ------------------------------------------------------------------------------------------------ one pass
def _own(s):
    c = s["case"]
    if c["op"] == "act8":
        from mixture_experts_layer_histogram_gb300 import _lib as L
        L.moe_act8_quantize(s["x"], s["codes"], s["scales"])
        L.moe_act8_dequantize(s["codes"], s["scales"], s["values"])
        return {"values": s["values"]}
    if c["op"] == "layernorm":
        norm = s["norm"]
        if c["dir"] == "bwd":
            return norm.backward(s["dn"], s["w"], x=s["x"], dx_in=s["dres"])
        res = {"n": norm.forward(s["x"], s["w"], s["b"])}
        if c["dir"] == "kept":
            res["again"] = norm.restore(s["w"], s["b"], out=s["again"])
            res.update(norm.backward(s["dn"], s["w"], dx_in=s["dres"]))
        return res
    ffn = s["ffn"]
    res = {"y": ffn.forward(s["x"], s["wgu"], s["wd"], add=s["add"])}
    if c["dir"] == "step":
        res.update(ffn.backward(s["dy"], s["x"], s["wgu"], s["wd"], add=s["dadd"]))
    return res


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "layernorm":
        return _plain_layernorm(state)
    if op == "ffn":
        return _plain_ffn(state)
    return {"values": _round8(state["x"].float()).to(state["x"].dtype)}


def work(case):
    c, z = case, 2 if case["dtype"] == "bf16" else 4
    if c["op"] == "act8":
        n = c["R"] * c["K"]
        return {"bytes": n * (2 * z + 2 * 33 / 32), "flops": 4 * n}
    if c["op"] == "layernorm":
        n, vecs = c["T"] * c["d"], (1 + c["bias"]) * c["d"] * z
        if c["dir"] == "fwd":
            return {"bytes": 2 * n * z + vecs, "flops": 8 * n}
        if c["dir"] == "bwd":
            return {"bytes": 4 * n * z + 2 * vecs + 8 * c["T"], "flops": 14 * n}
        return {"bytes": 6 * n * z + 3 * n * 33 / 32 + 3 * vecs + 4 * c["T"], "flops": 30 * n}   # forward; restored; backward
    T, d, f = c["T"], c["d"], c["f"]
    rows = 2 + c["add"]                                       # x, y, and what y adds to
    flops, moved = 6 * T * d * f, 3 * d * f * z + rows * T * d * z
    if c["dir"] == "step":
        kept = 2 * T * f * (33 / 32 if c["keep"] == "f8" else z)
        flops, moved = 3 * flops, 3 * 3 * d * f * z + (2 * rows + 1) * T * d * z + 2 * kept
    return {"bytes": moved, "flops": flops}


# ------------------------------------------------------------------------------------------------ in 64 bits
def _exact_round8(x):
    """The 8-bit values of x [R, K] in 64 bits: each magnitude against the midpoints between the 127 values of e4m3."""
    R, K = x.shape
    nb = -(-K // 32)
    b = torch.zeros(R, nb * 32, dtype=torch.float64, device=x.device)
    b[:, :K] = x
    b = b.view(R, nb, 32)
    e = torch.full((R, nb, 1), -127.0, dtype=torch.float64, device=x.device)
    top = b.abs().max(2, keepdim=True).values
    guess = torch.floor(torch.log2(top.clamp_min(2.0 ** -300) / 448))     # the logarithm may be off by one
    for k in (-1, 0, 1, 2):
        e = torch.where((e < guess + k) & (448 * torch.exp2((guess + k - 1)) < top), guess + k, e)
    e = e.clamp_min(-127)
    scale = torch.exp2(e)
    codes = torch.arange(127, dtype=torch.float64, device=x.device)
    grid = torch.where(codes < 8, codes * 2.0 ** -9, (8 + codes % 8) * torch.exp2(torch.floor(codes / 8) - 10))
    mid, a = (grid[1:] + grid[:-1]) / 2, (b / scale).abs()
    at = torch.searchsorted(mid, a.contiguous())                          # midpoints below a
    tie = mid[at.clamp_max(125)] == a                                     # half-way: to the even code
    at = torch.where(tie & (at % 2 == 1), at + 1, at)
    return (torch.sign(b) * grid[at] * scale).view(R, nb * 32)[:, :K]


def _exact_layernorm(s):
    c = s["case"]
    x, w = s["x"].double(), s["w"].double()
    if c["dir"] == "bwd":
        mean, sd = s["mean"].double()[:, None], 1 / s["rstd"].double()[:, None]
    else:
        mean = x.sum(1, keepdim=True) / c["d"]
        sd = ((x * x).sum(1, keepdim=True) / c["d"] - mean * mean + EPS).sqrt()
    z, res = (x - mean) / sd, {}

    def affine(v):
        return torch.addcmul(s["b"].double(), v, w) if c["bias"] else v * w

    if c["dir"] != "bwd":
        res["n"] = affine(z)
        if c["dir"] == "fwd":
            return res
        z = _exact_round8(z)
        res["again"] = affine(z)
    dn = s["dn"].double()
    inner = torch.einsum("td,d->t", dn, w)[:, None] / c["d"]
    along = torch.einsum("td,d,td->t", dn, w, z)[:, None] / c["d"]
    res["dx"] = s["dres"].double() + (dn * w - inner - along * z) / sd
    res["dw"] = torch.einsum("td,td->d", dn, z)
    if c["bias"]:
        res["db"] = torch.einsum("td->d", dn)
    return res


def _exact_ffn(s):
    c, f = s["case"], s["case"]["f"]
    x, wg, wu, wd = s["x"].double(), s["wgu"][:f].double(), s["wgu"][f:].double(), s["wd"].double()
    a, b = torch.einsum("td,fd->tf", x, wg), torch.einsum("td,fd->tf", x, wu)

    def arg(v):   # act(v) = v sigmoid(arg(v))
        return v if c["act"] == "silu" else 2 * GELU_C * (v + GELU_K * v ** 3)

    h = a * torch.sigmoid(arg(a)) * b
    res = {"y": torch.einsum("tf,df->td", h, wd)}
    if c["add"]:
        res["y"] = res["y"] + s["add"].double()
    if c["dir"] == "fwd":
        return res
    if c["keep"] == "f8":
        a, b = (_exact_round8(v) if f % 32 == 0 else None for v in (a, b))
    sg = torch.sigmoid(arg(a))
    slope = torch.ones_like(a) if c["act"] == "silu" else 2 * GELU_C * (1 + 3 * GELU_K * a ** 2)
    dy = s["dy"].double()
    dh = torch.einsum("td,df->tf", dy, wd)
    da, db = dh * b * (sg + a * sg * (1 - sg) * slope), dh * a * sg
    dx = torch.einsum("tf,fd->td", da, wg) + torch.einsum("tf,fd->td", db, wu)
    res["dx"] = dx + s["dadd"].double() if c["add"] else dx
    res["dw_gate_up"] = torch.cat([torch.einsum("tf,td->fd", da, x), torch.einsum("tf,td->fd", db, x)])
    res["dw_down"] = torch.einsum("td,tf->df", dy, a * sg * b)
    return res


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "layernorm":
        return _exact_layernorm(s)
    if case["op"] == "ffn":
        return _exact_ffn(s)
    return {"values": _exact_round8(s["x"])}
