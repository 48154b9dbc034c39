"""One MoE block trained and then served: norms, layer, optimiser and MXFP4 experts together.

    python examples/block_train_serve.py [--tokens 1024] [--steps 60] [--state f8|f32]

The block is  n = rms-norm(x),  y = MoE(n),  out = x + gate * rms-norm(y).  It learns a fixed random map of its
input under a squared error: BlockNorms and MoELayer give the gradients, one AdamW step updates every
parameter (8-bit states by default), all of it captured into one CUDA graph and replayed. The trained experts are
then quantised to MXFP4 and the same block runs on them.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from mixture_experts_layer_histogram_gb300 import AdamW, BlockNorms, Fp4Weights, MoELayer, MoELayerFp4  # noqa: E402


class Block:
    def __init__(self, T, d, E, k, f, state="f8", lr=3e-3, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        def randn(*shape, scale):
            return (torch.randn(shape, generator=g, device="cuda") * scale).bfloat16()
        self.T, self.d = T, d
        self.w_pre = torch.ones(d, dtype=torch.bfloat16, device="cuda")
        self.w_post = torch.ones(d, dtype=torch.bfloat16, device="cuda")
        self.gate = torch.full((d,), 0.5, dtype=torch.bfloat16, device="cuda")
        self.w_router = randn(E, d, scale=0.02)
        self.w_gate_up = randn(E, 2 * f, d, scale=0.02)
        self.w_down = randn(E, d, f, scale=0.02)
        self.norms = BlockNorms(T, d, torch.bfloat16, gate="channel", next_norm=False)
        self.layer = MoELayer(T, d, E, k, f, torch.bfloat16, router=True)
        self.dout = torch.empty((T, d), dtype=torch.bfloat16, device="cuda")
        self.loss = torch.zeros((), device="cuda")
        n, m = self.norms, self.layer
        self.opt = AdamW([self.w_pre, self.w_post, self.gate, self.w_router, self.w_gate_up, self.w_down],
                         [n.dw, n.dw_post, n.d_gate, m.dw_router, m.dw_gate_up, m.dw_down], lr=lr,
                         weight_decay=[0.0, 0.0, 0.0, 0.0, 0.01, 0.01], state=state)

    def forward(self, x):
        n = self.norms.pre(x, self.w_pre)
        self.y = self.layer.forward(n, None, self.w_gate_up, self.w_down, w_router=self.w_router)
        return self.norms.post(self.y, x, self.w_post, gate=self.gate)[0]

    def step(self, x, target):
        out = self.forward(x)
        diff = out.float() - target.float()
        self.loss.copy_((diff * diff).mean())
        self.dout.copy_(diff * (2.0 / diff.numel()))
        post = self.norms.post_backward(self.dout, None, None, self.y, self.w_post, gate=self.gate)
        dn = self.layer.backward(post["dy"], self.w_gate_up, self.w_down)["dx"]
        self.norms.pre_backward(dn, x, self.w_pre, dx_in=post["dx"])   # adds to post's dx in its place
        self.opt.step()

    def serve(self):
        """The block's forward with its experts in MXFP4, as a function of x."""
        m = self.layer
        fp4 = MoELayerFp4(self.T, self.d, m.E, m.k, m.f)
        weights = Fp4Weights.quantize(self.w_gate_up, self.w_down)

        def run(x):
            n = self.norms.pre(x, self.w_pre)
            logits = n.float() @ self.w_router.float().T
            y = fp4.forward(n, logits, weights)
            return self.norms.post(y, x, self.w_post, gate=self.gate)[0]
        return run


def main(tokens=1024, steps=60, state="f8", d=512, E=8, k=2, f=512):
    torch.manual_seed(0)
    block = Block(tokens, d, E, k, f, state)
    x = torch.randn(tokens, d, device="cuda").bfloat16()
    target = (x.float() + torch.tanh(x.float() @ (torch.randn(d, d, device="cuda") / d ** 0.5))).bfloat16()
    block.step(x, target)                                    # first step outside the capture
    first = block.loss.item()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        block.step(x, target)
    for _ in range(steps - 1):
        graph.replay()
    last = block.loss.item()
    out = block.forward(x).clone()
    served = block.serve()(x)
    move, err = (out.float() - x.float()).norm().item(), (served.float() - out.float()).norm().item()
    print(f"loss {first:.4f} -> {last:.4f} in {block.opt.steps} steps; "
          f"MXFP4 experts change the block's update of the stream by {100 * err / move:.1f} %")
    return first, last, err / move


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=1024)
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--state", choices=("f8", "f32"), default="f8")
    a = ap.parse_args()
    main(a.tokens, a.steps, a.state)
