"""The gated feed-forward block, y = (act(x Wg^T) * (x Wu^T)) Wd^T: the expert that every token takes. Beside a MoELayer it
adds to the routed experts' output in its place, in a dense block it stands alone.

    ffn = GatedFFN(T, d, f)                                     # training; backward=False: inference
    y = ffn.forward(x, w_gate_up, w_down, add=layer_out)        # w_gate_up [2f, d]: gate rows first; w_down [d, f]
    grads = ffn.backward(dy, x, w_gate_up, w_down, add=dx)      # dx, dw_gate_up, dw_down

keep="f8" keeps the gate and up projections in 8 bits between forward and backward (33 bytes per 32 values, and no h)
instead of in bf16.
"""
from __future__ import annotations

import torch

from . import _lib as L

ACTS = {"silu": L.ACT_SILU, "gelu": L.ACT_GELU}


class GatedFFN(L.OwnsBuffers):
    """Buffers of one block, allocated once and reused every step. Another tensor of the same type and shape may be set in the place
    of any of them (y, h, ab, ab_scales, dab, dx, dw_gate_up, dw_down; ws: zeros)."""

    _buffers = frozenset(("y", "h", "ab", "ab_scales", "dab", "dx", "dw_gate_up", "dw_down", "ws"))
    _fixed = frozenset(("T", "d", "f", "dtype", "device", "act", "keep", "backward_enabled"))

    def __init__(self, T, d, f, dtype=torch.bfloat16, act="silu", keep=None, backward=True, scratch=None, device="cuda"):
        """act: "silu" or "gelu" (its tanh form). keep: None (everything the backward reads, in dtype) or "f8". scratch: a
        dict with "h" [T, f] and "dab" [T, 2f] in dtype, shared with other blocks: dab always may be, h with keep="f8" or
        without a backward."""
        if act not in ACTS:
            raise ValueError(f"act is one of {sorted(ACTS)}, got {act!r}")
        if keep not in (None, "f8"):
            raise ValueError(f"keep is None or 'f8', got {keep!r}")
        if keep and not backward:
            raise ValueError("keep needs a backward")
        ws_bytes = L.moe_ffn_workspace_size(T, d, f, L.dtype_code(dtype), backward)
        if ws_bytes == 0:
            raise ValueError(f"GatedFFN takes T from 0 to {L.FFN_MAX_T} and d, f from 1 to {L.FFN_MAX}, in bfloat16 multiples of 8, got "
                             f"T = {T}, d = {d}, f = {f} in {dtype}")
        if keep and (dtype != torch.bfloat16 or f % 32):
            raise ValueError(f"keep='f8' is for bfloat16 and f a multiple of 32, got {dtype}, f = {f}")
        if not torch.cuda.is_available():
            raise RuntimeError("GatedFFN needs a CUDA device")
        self.T, self.d, self.f, self.dtype, self.act, self.keep = T, d, f, dtype, act, keep
        self.device = torch.device(device)
        self._act = ACTS[act]
        scratch = scratch or {}
        if "h" in scratch and backward and not keep:
            raise ValueError("without keep the backward reads h: it cannot be shared")
        act_ = dict(dtype=dtype, device=self.device)
        u8 = dict(dtype=torch.uint8, device=self.device)
        for name, shape in (("h", (T, f)), ("dab", (T, 2 * f))):
            if name in scratch:
                L._want(f"scratch[{name!r}]", scratch[name], dtype, shape)
                if scratch[name].device != torch.empty(0, **act_).device:
                    raise ValueError(f"scratch[{name!r}] is on {scratch[name].device}, the block is on {self.device}")
        self.h = scratch["h"] if "h" in scratch else torch.empty((T, f), **act_)
        self.y = torch.empty((T, d), **act_)
        self.ws = torch.zeros(ws_bytes, **u8)
        self.ab = self.ab_scales = None
        self.backward_enabled = backward
        if backward:
            if keep:
                self.ab = torch.empty((T, 2 * f), **u8)
                self.ab_scales = torch.empty(L.moe_act8_scale_bytes(T, 2 * f), **u8)
            else:
                self.ab = torch.empty((T, 2 * f), **act_)
            self.dab = scratch["dab"] if "dab" in scratch else torch.empty((T, 2 * f), **act_)
            self.dx = torch.empty((T, d), **act_)
            self.dw_gate_up = torch.empty((2 * f, d), **act_)
            self.dw_down = torch.empty((d, f), **act_)
        self._built()

    def _take(self):
        self._index = self.y.device.index
        with torch.cuda.device(self._index):
            self._kept = L.kept(self.ab, self.ab_scales, self.dtype, self.T, self.f)
        if self.backward_enabled:
            self._grads = [t.data_ptr() for t in (self.dab, self.dx, self.dw_gate_up, self.dw_down)]
        self._h_ptr, self._y_ptr, self._ws_ptr, self._ws_bytes = (self.h.data_ptr(), self.y.data_ptr(), self.ws.data_ptr(),
                                                                  self.ws.numel())

    def forward(self, x, w_gate_up, w_down, add=None, out=None, stream=None):
        """y [T, d] = add + FFN(x), into `out` (which may be add) where it is given."""
        dev = L._device()
        if dev != self._index:
            L.wrong_device(self._index, dev)
        y = self._y_ptr if out is None else L._at("out", out, self.dtype, (self.T, self.d), dev)
        L.ffn_fwd_into(dev, x, w_gate_up, w_down, add, self.T, self.d, self.f, self.dtype, self._act, self._kept, self._h_ptr, y,
                       self._ws_ptr, self._ws_bytes, stream)
        return self.y if out is None else out

    def backward(self, dy, x, w_gate_up, w_down, add=None, stream=None):
        """Gradients from what the last forward kept and its x: dx = add + the block's, dw_gate_up, dw_down."""
        if not self.backward_enabled:
            raise RuntimeError("the block was built without backward buffers")
        dev = L._device()
        if dev != self._index:
            L.wrong_device(self._index, dev)
        L.ffn_bwd_into(dev, dy, x, w_gate_up, w_down, add, self.T, self.d, self.f, self.dtype, self._act, self._kept, self._h_ptr,
                       *self._grads, self._ws_ptr, self._ws_bytes, stream)
        return dict(dx=self.dx, dw_gate_up=self.dw_gate_up, dw_down=self.dw_down)

    def status(self, stream=None):
        """Device status word (synchronises). After an error the workspace has to be zeroed before the next call: ws.zero_()."""
        return L.moe_read_status(self.ws, stream)
