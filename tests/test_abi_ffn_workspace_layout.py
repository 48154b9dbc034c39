"""Where the gated feed-forward block's workspace has its counts and its parts does not depend on the number of tokens, so that one
may serve calls of any (no GPU needed)."""
import os

import pytest

BF16 = 1


@pytest.fixture(scope="module")
def size():
    from mixture_experts_layer_histogram_gb300 import _lib, build
    if not os.path.exists(_lib.LIB_PATH):
        build.build()
    return _lib.lib().moe_ffn_workspace_size


@pytest.mark.parametrize("backward", [0, 1])
def test_counts_take_the_same_room_for_every_number_of_tokens(size, backward):
    """Every product (weight gradients of 4096 x 4096 too: 256 tiles of 256 x 256) has more tiles than the GPU's 76 pairs of SMs, so none
    is cut: what is left of the size is the counts."""
    assert len({size(T, 4096, 4096, BF16, backward) for T in (0, 20000, 40000, 100000, 1 << 20, 1 << 22)}) == 1


def test_parts_lie_behind_them(size):
    parts = 16 * 32 * 128 * 4                        # bytes of a part: 16 slices of 32 x 128 sums
    for T, d, f in ((389, 2048, 1024), (1, 8192, 8192), (255, 72, 6752)):
        more = size(T, d, f, BF16, 1) - size(0, d, f, BF16, 1)
        assert more > 0 and more % parts == 0
