"""Sizes past 32 bits: refused by the binding, where ctypes would hand the library their low bits (no GPU needed: tensors without
storage that claim to be on one)."""
import os

import pytest
import torch

from test_abi_activations import B, Claimed   # noqa: F401  (a fixture)

BF, U8 = torch.bfloat16, torch.uint8
LARGE = 2 ** 32 + 64                 # its low bits are 64


class Bare(Claimed):
    def __init__(self, *shape, dtype=BF):
        self._t, self.is_cuda, self._dev = torch.empty(shape, dtype=dtype, device="meta"), True, 0


def test_act8(B):   # noqa: F811
    L, calls = B
    for shape in ((LARGE,), (1, LARGE), (2, 3, 2 ** 31)):
        x, codes, scales = Bare(*shape), Bare(*shape, dtype=U8), Bare(2 ** 40, dtype=U8)
        for call in (lambda: L.moe_act8_quantize(x, codes, scales), lambda: L.moe_act8_dequantize(codes, scales, x)):
            with pytest.raises(ValueError, match="past 2"):
                call()
    assert calls == []
    # rows may be many: their number has 64 bits
    L.moe_act8_quantize(Bare(LARGE, 32), Bare(LARGE, 32, dtype=U8), Bare(LARGE, dtype=U8))
    assert calls[-1][1][2:4] == (LARGE, 32)


def test_layer_norm(B):   # noqa: F811
    L, calls = B
    f32 = torch.float32
    for T, d in ((LARGE, 8), (1, LARGE), (2 ** 31, 1)):
        rows, vec, stat, codes, scales = Bare(T, d), Bare(d), Bare(T, dtype=f32), Bare(T, d, dtype=U8), Bare(2 ** 40, dtype=U8)
        for call in (lambda: L.moe_layer_norm_fwd(rows, vec, vec, rows, stat, stat), lambda: L.moe_layer_norm_restore(codes, scales, vec, None, rows),
                     lambda: L.moe_layer_norm_bwd(rows, rows, None, None, stat, stat, vec, None, rows, vec, vec, Bare(64, dtype=U8))):
            with pytest.raises(ValueError, match="past 2"):
                call()
    assert calls == []


def test_ffn(B):   # noqa: F811
    L, calls = B
    for T, d, f in ((LARGE, 8, 8), (4, LARGE, 8), (4, 8, LARGE)):
        x, wgu, wd, h, dab = Bare(T, d), Bare(2 * f, d), Bare(d, f), Bare(T, f), Bare(T, 2 * f)
        ws = Bare(2 ** 40, dtype=U8)
        for call in (lambda: L.moe_ffn_fwd(x, wgu, wd, None, None, None, h, x, ws),
                     lambda: L.moe_ffn_bwd(x, x, dab, None, h, wgu, wd, None, dab, x, wgu, wd, ws)):
            with pytest.raises(ValueError, match="past 2"):
                call()
    assert calls == []


def test_sizes_of_buffers():
    from mixture_experts_layer_histogram_gb300 import GatedFFN, LayerNorm
    from mixture_experts_layer_histogram_gb300 import _lib as L, build
    if not os.path.exists(L.LIB_PATH):
        build.build()
    for call in (lambda: L.moe_act8_scale_bytes(4, LARGE), lambda: L.moe_layer_norm_bwd_workspace_size(LARGE, 64, 1),
                 lambda: L.moe_layer_norm_bwd_workspace_size(4, LARGE, 1), lambda: L.moe_ffn_workspace_size(LARGE, 64, 64, 1, True),
                 lambda: L.moe_ffn_workspace_size(4, LARGE, 64, 1, True), lambda: L.moe_ffn_workspace_size(4, 64, LARGE, 1, True),
                 lambda: LayerNorm(LARGE, 64), lambda: LayerNorm(4, LARGE, backward=False), lambda: GatedFFN(4, 64, LARGE, backward=False)):
        with pytest.raises(ValueError, match="past 2"):
            call()
    assert L.moe_act8_scale_bytes(LARGE, 64) == 2 * LARGE
