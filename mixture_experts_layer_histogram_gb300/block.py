"""Norms around one block: the RMS norm before it, and after it the norm of the block's output fused with
its gate, the scaled residual and the next block's norm.

  n        = x rms(x) w                                    pre
  out      = res_scale x + gate * (y rms(y) w_post)        post: y is the block's output
  n_next   = out rms(out) w_next                           (in the same pass)

A stack of blocks calls pre once, then post after every block, which leaves the stream and the next
block's input; the backward calls post_backward from the last block to the first (dx of one is dout of
the one before) and pre_backward at the bottom.
"""
from __future__ import annotations

import torch

from . import _lib as L


class BlockNorms:
    """Buffers of one block's norms, allocated once and reused every step."""

    def __init__(self, T, d, dtype=torch.bfloat16, gate=None, res_scale=1.0, eps=1e-6, next_norm=True, backward=True,
                 device="cuda"):
        """gate: None, "channel" (gate [d]) or "token" (gate [T, d]). next_norm: post also norms the stream for
        the next block."""
        if gate not in (None, "channel", "token"):
            raise ValueError(f"gate is None, 'channel' or 'token', got {gate!r}")
        if not torch.cuda.is_available():
            raise RuntimeError("BlockNorms needs a CUDA device")
        self.T, self.d, self.dtype, self.gate_kind = T, d, dtype, gate
        self.res_scale, self.eps, self.next_norm = res_scale, eps, next_norm
        self.device = torch.device(device)
        act = dict(dtype=dtype, device=self.device)
        self.n_first = torch.empty((T, d), **act)      # pre's output: the block may read it again in its backward
        self.n = torch.empty((T, d), **act) if next_norm else None
        self.out = torch.empty((T, d), **act)
        self._kind = {None: L.GATE_NONE, "channel": L.GATE_CHANNEL, "token": L.GATE_TOKEN}[gate]
        self._out_ptr, self._n_ptr = self.out.data_ptr(), self.n.data_ptr() if next_norm else None
        code = L.dtype_code(dtype)
        self.backward_enabled = backward
        if backward:
            self.dx = torch.empty((T, d), **act)
            self.dy = torch.empty((T, d), **act)
            self.dw = torch.empty(d, **act)
            self.dw_post = torch.empty(d, **act)
            self.dw_next = torch.empty(d, **act) if next_norm else None
            self.d_gate = None if gate is None else torch.empty((d,) if gate == "channel" else (T, d), **act)
            self.ws = torch.empty(L.moe_norm_bwd_workspace_size(T, d, code), dtype=torch.uint8, device=self.device)

    def _check_gate(self, gate):
        have = None if gate is None else ("channel" if gate.dim() == 1 else "token")
        if have != self.gate_kind:
            raise ValueError(f"built for gate {self.gate_kind!r}, got {have!r}")

    def pre(self, x, w, stream=None):
        """n [T, d] = x rms(x) w."""
        L.moe_norm_fwd(x, w, self.n_first, self.eps, stream)
        return self.n_first

    def post(self, y, x, w_post, gate=None, w_next=None, stream=None):
        """(out, n): the stream after the block and the next block's input (None without a next norm)."""
        if (w_next is not None) != self.next_norm:
            raise ValueError("w_next is needed with a next norm, and only there")
        if self._kind or gate is not None:
            self._check_gate(gate)
        L.norm_residual_fwd_into(y, x, w_post, gate, self._kind, w_next, self.T, self.d, self.dtype, self._out_ptr,
                                 self._n_ptr, self.res_scale, self.eps, stream)
        return self.out, self.n

    def post_backward(self, dout, dn, out, y, w_post, gate=None, w_next=None, stream=None):
        """Gradients of post: dout reaches out through the stream, dn through the next norm. Returns dx, dy, dw_post,
        and d_gate and dw_next where there are such."""
        if not self.backward_enabled:
            raise RuntimeError("norms were built without backward buffers")
        self._check_gate(gate)
        L.moe_norm_residual_bwd(dout, dn, out, y, w_post, gate, w_next, self.dx, self.dy, self.dw_post, self.d_gate,
                                self.dw_next, self.ws, self.res_scale, self.eps, stream)
        res = dict(dx=self.dx, dy=self.dy, dw_post=self.dw_post)
        if gate is not None:
            res["d_gate"] = self.d_gate
        if w_next is not None:
            res["dw_next"] = self.dw_next
        return res

    def pre_backward(self, dn, x, w, dx_in=None, stream=None):
        """Gradients of pre: dx (plus dx_in, the gradient that reaches x through the residual) and dw."""
        if not self.backward_enabled:
            raise RuntimeError("norms were built without backward buffers")
        L.moe_norm_bwd(dn, x, w, dx_in, self.dx, self.dw, self.ws, self.eps, stream)
        return dict(dx=self.dx, dw=self.dw)
