"""AdamW takes tensors of one GPU only, and steps on that GPU. (No GPU needed: the tensors only claim to be on one.)"""
import pytest
import torch

from mixture_experts_layer_histogram_gb300 import AdamW
from mixture_experts_layer_histogram_gb300 import _lib as L


class Claimed:
    """A CPU tensor that says it is on a CUDA device."""

    def __init__(self, n, dtype=torch.float32, device=0):
        self._t, self.is_cuda, self.device = torch.zeros(n, dtype=dtype), True, torch.device("cuda", device)

    def __getattr__(self, name):
        return getattr(self._t, name)


N = 300


def make(state, other):
    """Arguments of a bf16 parameter with a master; `other` lies on the second GPU."""
    b, f8 = torch.bfloat16, state == "f8"
    held = torch.float8_e4m3fn if f8 else torch.float32
    on = lambda name: 1 if name == other else 0   # noqa: E731
    a = dict(params=[Claimed(N, b), Claimed(N, b, on("params"))], grads=[Claimed(N, b), Claimed(N, b, on("grads"))],
             masters=[Claimed(N), Claimed(N, device=on("masters"))], m=[Claimed(N, held), Claimed(N, held, on("m"))],
             v=[Claimed(N, held), Claimed(N, held, on("v"))], state=state)
    if f8:
        a.update(m_scale=[Claimed(2), Claimed(2, device=on("m_scale"))], v_scale=[Claimed(2), Claimed(2, device=on("v_scale"))])
    return a


@pytest.mark.parametrize("state,other", [(s, o) for s in ("f32", "f8") for o in
                                         ("params", "grads", "masters", "m", "v") + (("m_scale", "v_scale") if s == "f8" else ())])
def test_a_tensor_on_another_gpu(state, other):
    with pytest.raises(ValueError, match="cuda:1"):
        AdamW(**make(state, other))


def test_states_given_on_another_gpu_than_the_parameter():
    a = make("f32", None)
    a["m"][0] = Claimed(N, device=1)
    with pytest.raises(ValueError, match="cuda:1"):
        AdamW(**a)


def test_a_step_with_another_current_gpu(monkeypatch):
    opt = AdamW.__new__(AdamW)
    opt._plan = opt._plan_device = opt._state = Claimed(8, torch.int64)
    opt.betas, opt.eps, opt._index = (0.9, 0.99), 1e-8, 0
    monkeypatch.setattr(L, "_device", lambda: 1)
    monkeypatch.setattr(L, "_raw_stream", lambda device: 0)
    with pytest.raises(ValueError, match="cuda:0"):
        opt.step()
