"""The gated feed-forward block without tokens at sizes where one token's products would be cut along K."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from mixture_experts_layer_histogram_gb300 import GatedFFN

BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("d,f,dtype,keep", [(2048, 1216, BF, None), (256, 8192, BF, "f8"), (72, 6752, BF, None), (72, 6753, F32, None)])
def test_no_tokens(d, f, dtype, keep):
    ffn = GatedFFN(0, d, f, dtype, keep=keep)
    e = torch.empty(0, d, dtype=dtype, device="cuda")
    wgu, wd = torch.ones(2 * f, d, dtype=dtype, device="cuda"), torch.ones(d, f, dtype=dtype, device="cuda")
    ffn.dw_gate_up.fill_(3)
    ffn.dw_down.fill_(3)
    assert ffn.forward(e, wgu, wd).shape == (0, d)
    res = ffn.backward(e, e, wgu, wd)
    assert res["dw_gate_up"].eq(0).all() and res["dw_down"].eq(0).all() and res["dx"].shape == (0, d) and ffn.status() == 0
