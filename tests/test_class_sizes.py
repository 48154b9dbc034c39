"""Sizes, types and eps that LayerNorm and GatedFFN refuse when they are built, not at their first call (no GPU needed)."""
import os

import pytest
import torch

from mixture_experts_layer_histogram_gb300 import GatedFFN, LayerNorm

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True, scope="module")
def built():
    from mixture_experts_layer_histogram_gb300 import _lib, build
    if not os.path.exists(_lib.LIB_PATH):
        build.build()


@pytest.mark.parametrize("args,kw", [((4, 60, 64), {}), ((4, 64, 60), {}), ((4, 0, 64), {}), ((4, 64, 0), {}), ((-1, 64, 64), {}),
                                     (((1 << 22) + 1, 64, 64), {}), ((4, (1 << 20) + 8, 64), {}), ((4, 64, (1 << 20) + 8), {}),
                                     ((4, 64, 40), dict(keep="f8")), ((4, 64, 64), dict(keep="f8", dtype=F32)), ((4, 0, 3), dict(dtype=F32))])
@pytest.mark.parametrize("backward", [True, False])
def test_ffn(args, kw, backward):
    if "keep" in kw and not backward:
        return
    with pytest.raises(ValueError, match="d = |multiple of 32"):
        GatedFFN(*args, backward=backward, **kw)


@pytest.mark.parametrize("args", [(4, 8193), (4, 9000), (4, 0), (-1, 64)])
@pytest.mark.parametrize("backward", [True, False])
def test_norm(args, backward):
    for dtype in (BF, F32):
        with pytest.raises(ValueError, match="rows of 1 to 8192"):
            LayerNorm(*args, dtype, backward=backward)


@pytest.mark.parametrize("eps", [0.0, -1e-5, float("nan")])
def test_eps(eps):
    with pytest.raises(ValueError, match="eps"):
        LayerNorm(4, 64, eps=eps)


def test_types():
    for make in (lambda: LayerNorm(4, 64, torch.float16), lambda: GatedFFN(4, 64, 64, torch.float16)):
        with pytest.raises(TypeError, match="float16"):
            make()


def test_limits_are_the_header_s():
    from mixture_experts_layer_histogram_gb300 import _lib as L
    size = L.moe_ffn_workspace_size
    for T, d, f in ((L.FFN_MAX_T, 8, 8), (1, L.FFN_MAX, 8), (1, 8, L.FFN_MAX)):
        assert size(T, d, f, L.MOE_BF16, True) > 0
    assert size(L.FFN_MAX_T + 1, 8, 8, L.MOE_BF16, True) == size(1, L.FFN_MAX + 8, 8, L.MOE_BF16, True) == 0
    assert L.moe_layer_norm_bwd_workspace_size(1, L.NORM_MAX_D, 1) > 0 == L.moe_layer_norm_bwd_workspace_size(1, L.NORM_MAX_D + 1, 1)
