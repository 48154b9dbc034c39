"""The gated feed-forward block's forward on both sides of the sizes at which few tokens change their path."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from mixture_experts_layer_histogram_gb300 import GatedFFN

    from test_gpu_ffn import BF, check_forward, make


@pytest.mark.parametrize("T,d,f", [(16, 4104, 8200), (17, 4104, 8200), (17, 4104, 2728), (32, 1000, 10248), (33, 1000, 10248), (33, 2056, 2120),
                                   (33, 2056, 2136), (64, 1000, 4104), (64, 520, 8400), (65, 520, 8400), (24, 2056, 8200), (48, 4104, 2056)])
def test_forward(T, d, f):
    check_forward(GatedFFN(T, d, f, act="gelu", backward=False), make(T, d, f, BF, T + d + f), "gelu", True)
