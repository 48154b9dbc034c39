"""Buffers that are set in the place of a class's own: taken where they fit, refused where they do not (no GPU needed: the layer norm's
buffers are put on the CPU, and only addresses are looked at)."""
import copy
import io
import os

import pytest
import torch

from mixture_experts_layer_histogram_gb300 import LayerNorm


@pytest.fixture
def made(monkeypatch):
    from mixture_experts_layer_histogram_gb300 import _lib, build
    if not os.path.exists(_lib.LIB_PATH):
        build.build()
    monkeypatch.setattr(torch.cuda, "is_available", lambda: True)
    return lambda **kw: LayerNorm(4, 64, device="cpu", **kw)


def test_calls_use_the_buffer_that_is_set(made):
    for keep in (None, "f8"):
        nm = made(keep=keep)
        for name in ("n", "codes" if keep else "mean", "rstd", "dx", "dw", "db", "ws"):
            old, new = getattr(nm, name), torch.empty_like(getattr(nm, name))
            where = [a.index(old.data_ptr()) if old.data_ptr() in a else None for a in (nm._out, nm._codes, nm._back)]
            assert any(i is not None for i in where)
            setattr(nm, name, new)
            assert getattr(nm, name) is new
            for i, a in zip(where, (nm._out, nm._codes, nm._back)):
                assert old.data_ptr() not in a and (i is None or a[i] == new.data_ptr()), name


def test_refusals(made):
    nm = made()
    before = [list(nm._out), list(nm._back)]
    for name, bad in (("n", torch.empty(4, 64)), ("n", torch.empty(5, 64, dtype=torch.bfloat16)), ("n", torch.empty(64, 4, dtype=torch.bfloat16).T),
                      ("mean", torch.empty(5)), ("mean", torch.empty(4, dtype=torch.float64)), ("n", torch.empty(4, 64, dtype=torch.bfloat16, device="meta")),
                      ("ws", torch.empty(8, dtype=torch.uint8)), ("n", None), ("codes", torch.empty(4, 64, dtype=torch.uint8))):
        with pytest.raises(ValueError, match=name):
            setattr(nm, name, bad)
    with pytest.raises(AttributeError, match="dx"):
        del nm.dx
    assert before == [nm._out, nm._back]
    nm = made(backward=False)
    with pytest.raises(ValueError, match="without"):
        nm.dx = torch.empty(4, 64, dtype=torch.bfloat16)
    nm.eps = 1e-3                                           # (no buffer)


@pytest.mark.parametrize("name,value", [("T", 5), ("T", 4), ("d", 32), ("dtype", torch.float32), ("bias", False), ("keep", "f8"),
                                        ("backward_enabled", False), ("device", torch.device("cpu"))])
def test_sizes_stay(made, name, value):
    """Calls check their inputs against these, and the buffers are as large as they said at the construction."""
    nm = made()
    with pytest.raises(AttributeError, match=name):
        setattr(nm, name, value)


def test_copies_use_their_own_buffers(made):
    nm = made(keep="f8")
    stream = io.BytesIO()
    torch.save(nm, stream)
    stream.seek(0)
    for other in (copy.deepcopy(nm), torch.load(stream, weights_only=False)):
        for mine, own in ((other._out, nm._out), (other._codes, nm._codes), (other._back, nm._back)):
            assert [p is None for p in mine] == [p is None for p in own] and not {p for p in mine if p} & {p for p in own if p}
        assert other._out[0] == other.n.data_ptr() and other._back[-1] == other.ws.data_ptr() and other._ws_bytes == nm._ws_bytes
    assert copy.copy(nm)._out == nm._out                    # a shallow copy shares them
