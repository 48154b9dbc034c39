"""Activations in 8 bits (e4m3 codes, one power of two per 32 values of a row): what a forward keeps for its backward in
about half the bytes of bf16.

    codes, scales = act8_quantize(x)                 # after the forward has used x
    x = act8_dequantize(codes, scales)               # before the backward needs it

LayerNorm(keep="f8") and GatedFFN(keep="f8") write and read this format themselves.
"""
from __future__ import annotations

import torch

from . import _lib as L


def act8_quantize(x, stream=None):
    """8-bit codes [..., K] (uint8) and scales of x [..., K]."""
    R, K = L._rows(x.shape)
    codes = torch.empty(x.shape, dtype=torch.uint8, device=x.device)
    scales = torch.empty(L.moe_act8_scale_bytes(R, K), dtype=torch.uint8, device=x.device)
    L.moe_act8_quantize(x, codes, scales, stream)
    return codes, scales


def act8_dequantize(codes, scales, dtype=torch.bfloat16, out=None, stream=None):
    """The values that the codes and scales stand for, [..., K], into `out` where it is given."""
    x = torch.empty(codes.shape, dtype=dtype, device=codes.device) if out is None else out
    L.moe_act8_dequantize(codes, scales, x, stream)
    return x
