"""AdamW over many tensors at once: one launch per kind of tensor, states in fp32 or in 8 bits.

    opt = AdamW([w_gate_up, w_down], [layer.dw_gate_up, layer.dw_down], lr=1e-4, state="f8")
    ...
    opt.step()          # reads the gradient buffers, updates parameters and states in place

The plan holds the tensors' addresses, so parameters and gradients keep their buffers between steps
(as MoELayer's do). The step count, the learning rate and the gradient scale live in device memory: a
step captured into a CUDA graph counts on when it is replayed, and follows lr and grad_scale.
"""
from __future__ import annotations

import torch

from . import _lib as L


class AdamW:
    def __init__(self, params, grads, lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01, state="f32",
                 masters=None, m=None, v=None, m_scale=None, v_scale=None, step=0):
        """params, grads: contiguous CUDA tensors, fp32 or bf16 (a gradient in its parameter's type). All tensors are on
        one GPU, which is the current one when step is called.
        weight_decay: one value, or one per tensor. state: "f32", or "f8" (e4m3 codes with one fp32 scale per
        256 values; v as the codes of its root; not for tensors that mix gradients over 2^18 apart within 256
        values). masters: True for fp32 copies of the bf16 parameters, or a list of them (None for fp32
        parameters). m, v, m_scale, v_scale, step: states to go on from (they are updated in place)."""
        if state not in ("f32", "f8"):
            raise ValueError(f"state is 'f32' or 'f8', got {state!r}")
        params, grads = list(params), list(grads)
        if len(params) != len(grads):
            raise ValueError(f"{len(params)} parameters and {len(grads)} gradients")
        decays = list(weight_decay) if isinstance(weight_decay, (list, tuple)) else [weight_decay] * len(params)
        if len(decays) != len(params):
            raise ValueError(f"{len(params)} parameters and {len(decays)} weight decays")
        self.params, self.grads, self.state = params, grads, state
        self.betas, self.eps = betas, eps
        dev = params[0].device if params else torch.device("cuda")
        f8 = state == "f8"
        held = torch.float8_e4m3fn if f8 else torch.float32
        blocks = [-(-p.numel() // L.ADAMW_BLOCK) for p in params]
        if masters is True:
            masters = [p.float() if p.dtype == torch.bfloat16 else None for p in params]
        self.masters = list(masters) if masters is not None else [None] * len(params)
        if len(self.masters) != len(params):
            raise ValueError(f"{len(params)} parameters and {len(self.masters)} masters")
        self.m = self._states("m", m, held)
        self.v = self._states("v", v, held)
        self.m_scale = self._scales("m_scale", m_scale, blocks) if f8 else None
        self.v_scale = self._scales("v_scale", v_scale, blocks) if f8 else None
        tensors = []
        for i, (p, g) in enumerate(zip(params, grads)):
            L.dtype_code(p.dtype)
            L._want(f"params[{i}]", p, p.dtype, p.shape)
            L._want(f"grads[{i}]", g, p.dtype, p.shape)
            if self.masters[i] is not None:
                L._want(f"masters[{i}]", self.masters[i], torch.float32, p.shape)
            a = L.AdamWTensor(n=p.numel(), weight_decay=decays[i], dtype=L.dtype_code(p.dtype),
                              state=L.ADAMW_F8 if f8 else L.ADAMW_F32)
            for name, t in (("p", p), ("g", g), ("master", self.masters[i]), ("m", self.m[i]), ("v", self.v[i]),
                            ("m_scale", self.m_scale[i] if f8 else None), ("v_scale", self.v_scale[i] if f8 else None)):
                if t is not None and not t.is_cuda:
                    raise ValueError("libmoe takes CUDA tensors only")
                if t is not None and t.device != dev:
                    raise ValueError(f"{name} of parameter {i} is on {t.device}, the first parameter on {dev}")
                setattr(a, name, None if t is None else t.data_ptr())
            tensors.append(a)
        self._plan = L.moe_adamw_plan(tensors)
        self._plan_device = self._plan.to(dev)
        # moe_adamw_state: step, lr, grad_scale, arrived
        self._state = torch.zeros(3, dtype=torch.int64, device=dev)
        self._state[0] = step
        self._index = self._state.device.index
        self._hyper = self._state[1:2].view(torch.float32)
        self._hyper.copy_(torch.tensor([lr, 1.0]))

    def _states(self, name, given, dtype):
        if given is None:
            return [torch.zeros(p.shape, dtype=dtype, device=p.device) for p in self.params]
        for i, (t, p) in enumerate(zip(given, self.params)):
            L._want(f"{name}[{i}]", t, dtype, p.shape)
        if len(given) != len(self.params):
            raise ValueError(f"{name}: {len(given)} tensors for {len(self.params)} parameters")
        return list(given)

    def _scales(self, name, given, blocks):
        if given is None:
            return [torch.zeros(b, dtype=torch.float32, device=p.device) for b, p in zip(blocks, self.params)]
        if len(given) != len(blocks):
            raise ValueError(f"{name}: {len(given)} tensors for {len(blocks)} parameters")
        for i, (t, b) in enumerate(zip(given, blocks)):
            L._want(f"{name}[{i}]", t, torch.float32, (b,))
        return list(given)

    def step(self, stream=None):
        if L._device() != self._index:
            raise ValueError(f"the tensors are on cuda:{self._index}, the current device is cuda:{L._device()}")
        L.moe_adamw_step(self._plan, self._plan_device, self.betas[0], self.betas[1], self.eps, self._state, stream)

    def set_lr(self, lr):
        """Takes effect with the next step on the current stream (also of a captured step)."""
        self._hyper[0] = lr

    def set_grad_scale(self, scale):
        """Gradients are multiplied by it (loss scaling, clipping): a number, or a CUDA tensor of one value."""
        self._hyper[1] = scale

    @property
    def steps(self):
        """Steps taken (synchronises)."""
        return int(self._state[0])
