"""The block example end to end: training with 8-bit and fp32 optimiser states lowers the loss, and the MXFP4 experts
serve the trained block. Bounds: the target is reachable to a good part (the loss has to fall to below two thirds);
three roundings to E2M1, each of about 0.1 of a value, on tokens, weights and h leave the update of the stream
within 40 %."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("state", ["f8", "f32"])
def test_example(state):
    spec = importlib.util.spec_from_file_location("block_train_serve", os.path.join(ROOT, "examples", "block_train_serve.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    first, last, change = m.main(tokens=512, steps=40, state=state)
    assert last < 2 / 3 * first
    assert change < 0.4
