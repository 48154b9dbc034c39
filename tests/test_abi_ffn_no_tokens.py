"""Workspace sizes of the gated feed-forward block for every number of tokens, none among them (no GPU needed)."""
import os

import pytest

F32, BF16 = 0, 1


@pytest.fixture(scope="module")
def size():
    from mixture_experts_layer_histogram_gb300 import _lib, build
    if not os.path.exists(_lib.LIB_PATH):
        build.build()
    return _lib.lib().moe_ffn_workspace_size


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("backward", [0, 1])
@pytest.mark.parametrize("d,f", [(8, 8), (64, 32), (2048, 1024), (2048, 1216), (2048, 8192), (72, 6752), (1 << 20, 1 << 20)])
def test_no_tokens(size, d, f, backward, dtype):
    assert 64 <= size(0, d, f, dtype, backward) <= size(1, d, f, dtype, backward)


@pytest.mark.parametrize("d,f", [(8, 8), (72, 6752), (2048, 8192), (8192, 32), (1 << 20, 8), (8, 1 << 20)])
def test_few_tokens(size, d, f):
    for T in (*range(1, 20), 63, 64, 65, 255, 256, 257, 1023, 1 << 20, 1 << 22):
        assert size(T, d, f, BF16, 1) >= size(T, d, f, BF16, 0) >= 64
