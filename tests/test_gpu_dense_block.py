"""The operators of a block together, as they are used: layer norm that keeps 8 bits, the routed experts and the expert that every
token takes (added in its place), the backward from what was kept, an AdamW step, in one captured and replayed graph; against
autograd in 64 bits on the same (kept) activations.

Tolerances are on whole tensors (2-norm): each of a chain of n independent roundings to bf16 is off by at most 2^-8 of a value, by
2^-8 / sqrt(3) on the average at worst (uniform in half a step), so a gradient after n of them by about sqrt(n / 3) 2^-8: the longest
chain here (n, h or a, b, dab, dy of the combine, dx, their sum, the norm's dx) has fewer than 12, 2^-7 in all."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from mixture_experts_layer_histogram_gb300 import AdamW, GatedFFN, LayerNorm, MoELayer, act8_dequantize

T, D, E, K, F, FS = 384, 256, 4, 2, 256, 512
BF = torch.bfloat16
TOL = 2.0 ** -7


class Block:
    """out = x + MoE(n) + FFN(n), n = layer norm of x, with 8 bits kept per normalised value and per projection of the FFN."""

    def __init__(self, keep, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        r = lambda *s, k=1.0: (torch.randn(s, generator=g, device="cuda") * k).to(BF)  # noqa: E731
        self.p = dict(w=(1 + 0.2 * r(D).float()).to(BF), b=r(D, k=0.2), wgu=r(E, 2 * F, D, k=D ** -0.5), wd=r(E, D, F, k=F ** -0.5),
                      sgu=r(2 * FS, D, k=D ** -0.5), sd=r(D, FS, k=FS ** -0.5))
        self.norm = LayerNorm(T, D, keep=keep)
        self.moe = MoELayer(T, D, E, K, F)
        self.ffn = GatedFFN(T, D, FS, keep=keep)
        self.keep, self.again = keep, torch.empty(T, D, dtype=BF, device="cuda")
        self.out = torch.empty(T, D, dtype=BF, device="cuda")
        self.dn = torch.empty(T, D, dtype=BF, device="cuda")

    def forward(self, x, logits):
        p = self.p
        n = self.norm.forward(x, p["w"], p["b"])
        y = self.moe.forward(n, logits, p["wgu"], p["wd"])
        y = self.ffn.forward(n, p["sgu"], p["sd"], add=y, out=y)          # the shared expert adds in place
        torch.add(x, y, out=self.out)
        return self.out

    def backward(self, x, dout):
        p = self.p
        # without what the forward kept the block needs n again (the routed experts read their own copy)
        n = self.norm.restore(p["w"], p["b"], out=self.again) if self.keep else self.norm.n
        routed = self.moe.backward(dout, p["wgu"], p["wd"])
        shared = self.ffn.backward(dout, n, p["sgu"], p["sd"], add=routed["dx"])
        norm = self.norm.backward(shared["dx"], p["w"], x=None if self.keep else x, dx_in=dout)
        return dict(dx=norm["dx"], w=norm["dw"], b=norm["db"], wgu=routed["dw_gate_up"], wd=routed["dw_down"], sgu=shared["dw_gate_up"],
                    sd=shared["dw_down"], logits=routed["d_logits"])




def expected(blk, x, logits, dout):
    """The block's output and gradients by autograd in 64 bits; where the block keeps 8 bits, its backward sees those."""
    p = {k: v.double().requires_grad_() for k, v in blk.p.items()}
    x, lg = x.double().requires_grad_(), logits.double().requires_grad_()
    m = x.mean(1, keepdim=True)
    z = (x - m) / ((x - m).square().mean(1, keepdim=True) + 1e-5).sqrt()
    n = z * p["w"] + p["b"]
    top, idx = lg.topk(K, 1)
    w = torch.softmax(top, 1)
    y = torch.zeros_like(x)
    for e in range(E):
        tok, slot = (idx == e).nonzero(as_tuple=True)
        ab = n[tok] @ p["wgu"][e].T
        h = torch.nn.functional.silu(ab[:, :F]) * ab[:, F:]
        y = y.index_add(0, tok, (h @ p["wd"][e].T) * w[tok, slot][:, None])
    ab = n @ p["sgu"].T
    y = y + (torch.nn.functional.silu(ab[:, :FS]) * ab[:, FS:]) @ p["sd"].T
    out = x + y
    out.backward(dout.double())
    return out.detach(), dict({k: v.grad for k, v in p.items()}, dx=x.grad, logits=lg.grad)


def off(got, exp):
    return ((got.double() - exp).norm() / exp.norm()).item()


def inputs(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    return (r(T, D) + 0.3).to(BF), r(T, E), r(T, D).to(BF)


@pytest.mark.parametrize("keep", [None, "f8"])
def test_output_and_gradients(keep):
    blk = Block(keep)
    x, logits, dout = inputs(1)
    out = blk.forward(x, logits).clone()
    got = {k: v.clone() for k, v in blk.backward(x, dout).items()}
    assert blk.ffn.status() == 0 and blk.moe.status() == (0, 0)
    ref, exp = expected(blk, x, logits, dout)
    assert off(out, ref) <= TOL
    for k in got:
        # 8 bits: a kept value is off by at most 2^-4, 2^-4 / sqrt(3) on the average at worst, in z (norm) and in a, b (FFN): three
        # such factors at most in a gradient
        assert off(got[k], exp[k]) <= (TOL if keep is None else TOL + 2.0 ** -4), (k, off(got[k], exp[k]))


def test_kept_values_are_what_the_backward_uses():
    """From the kept codes themselves the FFN's gradients are those of the formulas to bf16's roundings."""
    blk = Block("f8")
    x, logits, dout = inputs(2)
    blk.forward(x, logits)
    n = blk.norm.restore(blk.p["w"], blk.p["b"], out=blk.again).double()
    ab = act8_dequantize(blk.ffn.ab, blk.ffn.ab_scales, torch.float32).double()
    a, b = ab[:, :FS], ab[:, FS:]
    s = torch.sigmoid(a)
    dh = dout.double() @ blk.p["sd"].double()
    dab = torch.cat([dh * b * s * (1 + a * (1 - s)), dh * a * s], 1)
    got = blk.ffn.backward(dout, blk.again, blk.p["sgu"], blk.p["sd"])
    assert off(got["dx"], dab @ blk.p["sgu"].double()) <= TOL
    assert off(got["dw_gate_up"], dab.T @ n) <= TOL and off(got["dw_down"], dout.double().T @ (a * s * b)) <= TOL


@pytest.mark.parametrize("keep", [None, "f8"])
def test_captured_training_step(keep):
    """Forward, backward and an optimiser step in one graph, replayed: the eager steps' bits."""
    def build():
        blk = Block(keep)
        params = [blk.p[k] for k in ("w", "b", "wgu", "wd", "sgu", "sd")]
        grads = [blk.norm.dw, blk.norm.db, blk.moe.dw_gate_up, blk.moe.dw_down, blk.ffn.dw_gate_up, blk.ffn.dw_down]
        return blk, AdamW(params, grads, lr=1e-2, state="f32")

    def step(blk, opt, x, logits, dout):
        blk.forward(x, logits)
        blk.backward(x, dout)
        opt.step()

    x, logits, dout = inputs(3)
    (eager, eo), (graphed, go) = build(), build()
    step(eager, eo, x, logits, dout)
    step(graphed, go, x, logits, dout)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(graphed, go, x, logits, dout)
    for i in range(3):
        a, b, c = inputs(10 + i)
        x.copy_(a)
        logits.copy_(b)
        dout.copy_(c)
        graph.replay()
        step(eager, eo, x, logits, dout)
        assert torch.equal(eager.out, graphed.out) and all(torch.equal(eager.p[k], graphed.p[k]) for k in eager.p)
    assert eo.steps == go.steps == 4 and eager.ffn.status() == graphed.ffn.status() == 0


def test_two_blocks_on_two_streams():
    """Launches whose units wait for one another, on two streams at once, beside other work on a third: each takes the GPU in turn."""
    big = 2048
    r = lambda *s, k=1.0: (torch.randn(s, device="cuda") * k).to(BF)  # noqa: E731
    x, wgu, wd, dy = r(big, 512), r(2048, 512, k=0.05), r(512, 1024, k=0.03), r(big, 512)
    one, two, ref = (GatedFFN(big, 512, 1024) for _ in range(3))
    small = [GatedFFN(100, 512, 1024) for _ in range(3)]                 # tiles cut along K

    def run(f, s, stream=None):
        f.forward(x, wgu, wd, stream=stream)
        f.backward(dy, x, wgu, wd, stream=stream)
        s.forward(x[:100], wgu, wd, stream=stream)

    run(ref, small[2])
    streams = [torch.cuda.Stream() for _ in range(3)]
    for st in streams:
        st.wait_stream(torch.cuda.current_stream())
    m = torch.randn(2048, 2048, device="cuda")
    for _ in range(20):
        with torch.cuda.stream(streams[2]):
            torch.mm(m, m)
        run(one, small[0], streams[0])
        run(two, small[1], streams[1])
    torch.cuda.synchronize()
    for f in (one, two):
        assert f.status() == 0
        assert all(torch.equal(getattr(f, k), getattr(ref, k)) for k in ("y", "dx", "dw_gate_up", "dw_down"))
    assert all(s.status() == 0 and torch.equal(s.y, small[2].y) for s in small)
