"""Serving one MoE layer with its expert weights in MXFP4 (4-bit codes, one 8-bit scale per 32 values).

    weights = Fp4Weights.quantize(w_gate_up, w_down)      # once, from bf16 or fp32 weights
    layer = MoELayerFp4(T, d, E, k, f)
    out = layer.forward(x, logits, weights)

Forward of a step (one stream, no host synchronisation): moe_route_count_index, moe_permute_fp4 (each
token quantised once, written to its k grouped rows), moe_grouped_ffn_fwd_fp4, moe_combine_fwd.
"""
from __future__ import annotations

import torch

from . import _lib as L


def fp4_quantize(x, stream=None):
    """MXFP4 codes [..., K/2] and scales of x [..., K]."""
    R, K = L._rows(x.shape)
    codes = torch.empty(x.shape[:-1] + (K // 2,), dtype=torch.uint8, device=x.device)
    scales = torch.empty(L.moe_fp4_scale_bytes(R, K), dtype=torch.uint8, device=x.device)
    L.moe_fp4_quantize(x, codes, scales, stream)
    return codes, scales


def fp4_dequantize(codes, scales, dtype=torch.bfloat16, stream=None):
    """The values that the codes and scales stand for, [..., K]."""
    x = torch.empty(codes.shape[:-1] + (codes.shape[-1] * 2,), dtype=dtype, device=codes.device)
    L.moe_fp4_dequantize(codes, scales, x, stream)
    return x


class Fp4Weights:
    """One layer's expert weights in MXFP4: gate/up [E, 2f, d] and down [E, d, f], quantised along their last axis."""

    def __init__(self, gate_up, gate_up_scales, down, down_scales):
        self.gate_up, self.gate_up_scales, self.down, self.down_scales = gate_up, gate_up_scales, down, down_scales

    @classmethod
    def quantize(cls, w_gate_up, w_down, stream=None):
        return cls(*fp4_quantize(w_gate_up, stream), *fp4_quantize(w_down, stream))


class MoELayerFp4:
    """Buffers of one layer's forward with MXFP4 experts, allocated once and reused every step."""

    def __init__(self, T, d, E, k, f, device="cuda"):
        if not torch.cuda.is_available():
            raise RuntimeError("MoELayerFp4 needs a CUDA device")
        self.T, self.d, self.E, self.k, self.f = T, d, E, k, f
        self.device = torch.device(device)
        self.rows_max = R = L.moe_grouped_rows_max(T, k, E)
        i32 = dict(dtype=torch.int32, device=self.device)
        u8 = dict(dtype=torch.uint8, device=self.device)
        self.topk_idx = torch.empty((T, k), **i32)
        self.topk_w = torch.empty((T, k), dtype=torch.float32, device=self.device)
        self.counts = torch.empty(E, **i32)
        self.offsets = torch.empty(E + 1, **i32)
        self.tile_offsets = torch.empty(E + 1, **i32)
        self.row_of_slot = torch.empty(T * k, **i32)
        self.token_of_row = torch.empty(R, **i32)
        self.ws_index = torch.zeros(L.moe_count_index_workspace_size(T, k, E), **u8)
        self.ws_ffn = torch.zeros(L.moe_grouped_ffn_workspace_size(E, d, f, R, L.MOE_BF16, False), **u8)
        self.x_codes = torch.empty((R, d // 2), **u8)
        self.x_scales = torch.empty(L.moe_fp4_scale_bytes(R, d), **u8)
        self.h_codes = torch.empty((R, f // 2), **u8)
        self.h_scales = torch.empty(L.moe_fp4_scale_bytes(R, f), **u8)
        self.y_perm = torch.empty((R, d), dtype=torch.bfloat16, device=self.device)
        self.out = torch.empty((T, d), dtype=torch.bfloat16, device=self.device)

    def forward(self, x, logits, weights, stream=None):
        """x [T, d] bf16 or fp32, logits [T, E] fp32 -> out [T, d] bf16."""
        L._want("x", x, x.dtype, (self.T, self.d))
        L._want("logits", logits, torch.float32, (self.T, self.E))
        L.moe_route_count_index(logits, self.k, self.topk_idx, self.topk_w, self.counts, self.offsets,
                                self.tile_offsets, self.row_of_slot, self.token_of_row, self.ws_index, stream)
        L.moe_permute_fp4(x, self.k, self.E, self.row_of_slot, self.counts, self.tile_offsets, self.x_codes,
                          self.x_scales, stream)
        L.moe_grouped_ffn_fwd_fp4(self.x_codes, self.x_scales, weights.gate_up, weights.gate_up_scales, weights.down,
                                  weights.down_scales, self.tile_offsets, self.offsets, self.h_codes, self.h_scales,
                                  self.y_perm, self.ws_ffn, stream)
        L.moe_combine_fwd(self.y_perm, self.topk_w, self.row_of_slot, self.T, self.k, self.out, stream)
        return self.out

    def status(self, stream=None):
        """Device status words (synchronises): (count_index, grouped_ffn)."""
        return L.moe_read_status(self.ws_index, stream), L.moe_read_status(self.ws_ffn, stream)
