"""Index tensors and inputs that the MXFP4 calls refuse before anything is launched: another type, too few entries, strides,
another number of tokens than the layer's. (No GPU needed: the tensors only claim to be on one.)"""
import pytest
import torch

from mixture_experts_layer_histogram_gb300 import MoELayerFp4
from mixture_experts_layer_histogram_gb300 import _lib as L


class Claimed:
    """A CPU tensor that says it is a CUDA tensor."""

    def __init__(self, t):
        self._t = t

    def __getattr__(self, name):
        return True if name == "is_cuda" else getattr(self._t, name)


T, D, F, E, K = 5, 256, 256, 4, 2
R = 128 * E


def claimed(shape, dtype=torch.uint8):
    return Claimed(torch.zeros(shape, dtype=dtype))


def ints(n):
    return claimed(n, torch.int32)


def wrong(n):
    """Stand-ins for an int32 tensor of n entries."""
    return {"int64": claimed(n, torch.int64), "float": claimed(n, torch.float32), "short": ints(n - 1), "none": ints(0),
            "strides": Claimed(torch.zeros(2 * n, dtype=torch.int32)[::2]), "cpu": torch.zeros(n, dtype=torch.int32)}


KINDS = sorted(wrong(2))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("arg", ["row_of_slot", "counts", "tile_offsets"])
def test_permutation(arg, kind):
    a = dict(row_of_slot=ints(T * K), counts=ints(E), tile_offsets=ints(E + 1))
    a[arg] = wrong(a[arg].numel())[kind]
    with pytest.raises(ValueError, match=arg if kind != "cpu" else "CUDA"):
        L.moe_permute_fp4(claimed((T, D), torch.bfloat16), K, E, a["row_of_slot"], a["counts"], a["tile_offsets"],
                          claimed((R, D // 2)), claimed(R * D // 32))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("arg", ["tile_offsets", "offsets"])
def test_ffn(arg, kind):
    a = dict(tile_offsets=ints(E + 1), offsets=ints(E + 1))
    a[arg] = wrong(E + 1)[kind]
    with pytest.raises(ValueError, match=arg if kind != "cpu" else "CUDA"):
        L.moe_grouped_ffn_fwd_fp4(claimed((R, D // 2)), claimed(R * D // 32), claimed((E, 2 * F, D // 2)),
                                  claimed(E * 2 * F * D // 32), claimed((E, D, F // 2)), claimed(E * D * F // 32),
                                  a["tile_offsets"], a["offsets"], claimed((R, F // 2)), claimed(R * F // 32),
                                  claimed((R, D), torch.bfloat16), claimed(4096))


@pytest.mark.parametrize("x,logits", [((T + 1, D), (T, E)), ((T - 1, D), (T, E)), ((T, D + 256), (T, E)), ((T, D), (T + 1, E)),
                                      ((T, D), (T, E + 1)), ((T, D), (T, E, 1))])
def test_forward_with_other_sizes_than_the_layers(x, logits):
    layer = MoELayerFp4.__new__(MoELayerFp4)
    layer.T, layer.d, layer.E, layer.k, layer.f = T, D, E, K, F
    with pytest.raises(ValueError, match="x" if x != (T, D) else "logits"):
        layer.forward(claimed(x, torch.bfloat16), claimed(logits, torch.float32), None)


def test_forward_with_logits_of_another_type():
    layer = MoELayerFp4.__new__(MoELayerFp4)
    layer.T, layer.d, layer.E, layer.k, layer.f = T, D, E, K, F
    with pytest.raises(ValueError, match="logits"):
        layer.forward(claimed((T, D), torch.bfloat16), claimed((T, E), torch.bfloat16), None)
