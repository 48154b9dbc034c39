"""Activations in 8 bits (e4m3 codes, one power of two per 32 values of a row): what a forward keeps for its backward in
about half the bytes of bf16.

    codes, scales = act8_quantize(x)                 # after the forward has used x
    x = act8_dequantize(codes, scales)               # before the backward needs it

LayerNorm(keep="f8") and GatedFFN(keep="f8") write and read this format themselves.
"""
from __future__ import annotations

import contextlib

import torch

from . import _lib as L


def _on(stream):
    """What is allocated inside belongs to the stream whose kernel writes it: memory of the current stream's may still be in use
    there, by what was launched before."""
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


def act8_quantize(x, stream=None):
    """8-bit codes [..., K] (uint8) and scales of x [..., K] (made on `stream` where it is given, like its own tensors)."""
    R, K = L._rows(x.shape)
    with _on(stream):
        codes = torch.empty(x.shape, dtype=torch.uint8, device=x.device)
        scales = torch.empty(L.moe_act8_scale_bytes(R, K), dtype=torch.uint8, device=x.device)
    L.moe_act8_quantize(x, codes, scales, stream)
    return codes, scales


def act8_dequantize(codes, scales, dtype=torch.bfloat16, out=None, stream=None):
    """The values that the codes and scales stand for, [..., K], into `out` where it is given (else made on `stream`, as above)."""
    if out is None:
        with _on(stream):
            out = torch.empty(codes.shape, dtype=dtype, device=codes.device)
    L.moe_act8_dequantize(codes, scales, out, stream)
    return out
