"""Layer norm before a block, n = (x - mean) / sqrt(var + eps) * w + b, and its backward. (BlockNorms has the RMS norms.)

    norm = LayerNorm(T, d)
    n = norm.forward(x, w, b)
    grads = norm.backward(dn, w, x=x, dx_in=...)      # dx, dw, db

keep="f8" keeps the normalised rows in 8 bits instead of x and n: the backward of the block that reads n takes
norm.restore(w, b), and norm.backward needs no x.
"""
from __future__ import annotations

import torch

from . import _lib as L


class LayerNorm(L.OwnsBuffers):
    """Buffers of one norm, allocated once and reused every step. Another tensor of the same type and shape may be set in the place
    of any of them (n, mean, rstd, codes, scales, dx, dw, db, ws)."""

    _buffers = frozenset(("n", "mean", "rstd", "codes", "scales", "dx", "dw", "db", "ws"))
    _fixed = frozenset(("T", "d", "dtype", "device", "bias", "keep", "backward_enabled"))

    def __init__(self, T, d, dtype=torch.bfloat16, eps=1e-5, bias=True, keep=None, backward=True, device="cuda"):
        """bias: the norm has one (b is given to every call, and the backward returns db). keep: None, or "f8"."""
        if keep not in (None, "f8"):
            raise ValueError(f"keep is None or 'f8', got {keep!r}")
        if keep and not backward:
            raise ValueError("keep needs a backward")
        code = L.dtype_code(dtype)
        ws_bytes = L.moe_layer_norm_bwd_workspace_size(T, d, code)
        if ws_bytes == 0:
            raise ValueError(f"LayerNorm takes T >= 0 rows of 1 to {L.NORM_MAX_D} values, got T = {T}, d = {d}")
        if not eps > 0:
            raise ValueError(f"eps is above 0, got {eps}")
        if not torch.cuda.is_available():
            raise RuntimeError("LayerNorm needs a CUDA device")
        self.T, self.d, self.dtype, self.eps, self.bias, self.keep = T, d, dtype, eps, bias, keep
        self.device = torch.device(device)
        act = dict(dtype=dtype, device=self.device)
        self.n = torch.empty((T, d), **act)
        self.backward_enabled = backward
        self.mean = self.rstd = self.codes = self.scales = None
        if backward:
            f32, u8 = dict(dtype=torch.float32, device=self.device), dict(dtype=torch.uint8, device=self.device)
            self.rstd = torch.empty(T, **f32)
            if keep:
                self.codes = torch.empty((T, d), **u8)
                self.scales = torch.empty(L.moe_act8_scale_bytes(T, d), **u8)
            else:
                self.mean = torch.empty(T, **f32)
            self.dx = torch.empty((T, d), **act)
            self.dw = torch.empty(d, **act)
            self.db = torch.empty(d, **act) if bias else None
            self.ws = torch.empty(ws_bytes, **u8)
        self._built()

    def _take(self):
        self._index = self.n.device.index

        def at(*tensors):
            return [None if t is None else t.data_ptr() for t in tensors]

        self._out, self._codes = at(self.n, self.mean, self.rstd, self.codes, self.scales), at(self.codes, self.scales)
        if self.backward_enabled:
            self._back = at(self.codes, self.scales, self.mean, self.rstd, self.dx, self.dw, self.db, self.ws)
            self._ws_bytes = self.ws.numel()

    def _check(self, b):
        """The current device, on which the buffers have to be."""
        if (b is not None) != self.bias:
            raise ValueError("b is needed with a bias, and only there")
        dev = L._device()
        if dev != self._index:
            L.wrong_device(self._index, dev)
        return dev

    def forward(self, x, w, b=None, stream=None):
        """n [T, d]."""
        L.layer_norm_fwd_into(self._check(b), x, w, b, self.T, self.d, self.dtype, *self._out, self.eps, stream)
        return self.n

    def restore(self, w, b=None, out=None, stream=None):
        """n again, from the kept rows, into `out` (or n's own buffer)."""
        if not self.keep:
            raise RuntimeError("the norm keeps nothing to restore n from")
        dev = self._check(b)
        n = self._out[0] if out is None else L._at("out", out, self.dtype, (self.T, self.d), dev)
        L.layer_norm_restore_into(dev, *self._codes, w, b, self.T, self.d, self.dtype, n, stream)
        return self.n if out is None else out

    def backward(self, dn, w, x=None, dx_in=None, stream=None):
        """dx (plus dx_in, the gradient that reaches x past the norm), dw, and db with a bias. x is what forward read;
        with keep it is not needed."""
        if not self.backward_enabled:
            raise RuntimeError("the norm was built without backward buffers")
        if (x is None) != bool(self.keep):
            raise ValueError("x is needed without keep, and only there")
        dev = L._device()
        if dev != self._index:
            L.wrong_device(self._index, dev)
        L.layer_norm_bwd_into(dev, dn, x, w, dx_in, self.T, self.d, self.dtype, *self._back, self._ws_bytes, self.eps, stream)
        res = dict(dx=self.dx, dw=self.dw)
        if self.bias:
            res["db"] = self.db
        return res
