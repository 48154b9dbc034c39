"""The combine right behind the product that writes its rows, over and over: the results of inputs that take turns in one
layer's buffers are those that each has alone. (The combine is resident before that product has ended.)"""
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from mixture_experts_layer_histogram_gb300 import Fp4Weights, MoELayerFp4


@pytest.mark.parametrize("T,d,E,k,f", [(1, 512, 8, 2, 256), (40, 2048, 16, 8, 512), (2000, 1024, 8, 4, 512)])
def test_inputs_taking_turns(T, d, E, k, f):
    g = torch.Generator(device="cuda").manual_seed(T)
    w = Fp4Weights.quantize(torch.randn(E, 2 * f, d, generator=g, device="cuda") * 0.05,
                            torch.randn(E, d, f, generator=g, device="cuda") * 0.05)
    layer = MoELayerFp4(T, d, E, k, f)
    sets, alone = [], []
    for _ in range(3):
        sets.append((torch.randn(T, d, generator=g, device="cuda").bfloat16(), torch.randn(T, E, generator=g, device="cuda")))
        layer.y_perm.fill_(float("nan"))
        alone.append(layer.forward(*sets[-1], w).clone())
        torch.cuda.synchronize()
    assert not torch.equal(alone[0], alone[1])
    outs = []
    for i in range(60):
        outs.append((i % 3, layer.forward(*sets[i % 3], w).clone()))
    for i, out in outs:
        assert torch.equal(out, alone[i])
    assert layer.status() == (0, 0)
