"""Arguments that the norms, the optimiser step and the MXFP4 calls refuse on the host (no GPU needed)."""
import ctypes
import os

import pytest

FAKE = ctypes.c_void_p(1 << 20)   # never dereferenced: every call below fails validation first
ODD = ctypes.c_void_p((1 << 20) + 4)
NULL = None


@pytest.fixture(scope="module")
def L():
    from mixture_experts_layer_histogram_gb300 import _lib, build
    if not os.path.exists(_lib.LIB_PATH):
        build.build()
    return _lib.lib()


def test_norm_refusals(L):
    assert L.moe_norm_fwd(FAKE, FAKE, 4, 0, 0, 1e-6, FAKE, NULL) == -1
    assert L.moe_norm_fwd(FAKE, FAKE, -1, 64, 0, 1e-6, FAKE, NULL) == -1
    assert L.moe_norm_fwd(FAKE, FAKE, 4, 64, 2, 1e-6, FAKE, NULL) == -1
    assert L.moe_norm_fwd(FAKE, FAKE, 4, 64, 0, 0.0, FAKE, NULL) == -1
    assert L.moe_norm_fwd(FAKE, FAKE, 4, 64, 0, float("nan"), FAKE, NULL) == -1
    assert L.moe_norm_fwd(FAKE, FAKE, 4, 8193, 0, 1e-6, FAKE, NULL) == -2
    assert L.moe_norm_fwd(ODD, FAKE, 4, 64, 0, 1e-6, FAKE, NULL) == -1
    assert L.moe_norm_fwd(FAKE, NULL, 4, 64, 0, 1e-6, FAKE, NULL) == -1
    assert L.moe_norm_fwd(NULL, NULL, 0, 64, 0, 1e-6, NULL, NULL) == 0
    # gate kind, a missing gate, an n without w_next and the other way round
    assert L.moe_norm_residual_fwd(FAKE, FAKE, FAKE, FAKE, 3, NULL, 4, 64, 0, 1.0, 1e-6, FAKE, NULL, NULL) == -1
    assert L.moe_norm_residual_fwd(FAKE, FAKE, FAKE, NULL, 1, NULL, 4, 64, 0, 1.0, 1e-6, FAKE, NULL, NULL) == -1
    assert L.moe_norm_residual_fwd(FAKE, FAKE, FAKE, NULL, 0, NULL, 4, 64, 0, 1.0, 1e-6, FAKE, FAKE, NULL) == -1
    assert L.moe_norm_residual_fwd(FAKE, FAKE, FAKE, NULL, 0, FAKE, 4, 64, 0, 1.0, 1e-6, FAKE, NULL, NULL) == -1
    ws = L.moe_norm_bwd_workspace_size(4, 64, 0)
    assert ws >= 2 * 64 * 4
    assert L.moe_norm_bwd(FAKE, FAKE, FAKE, NULL, 4, 64, 0, 1e-6, FAKE, FAKE, FAKE, ws - 1, NULL) == -1
    assert L.moe_norm_bwd(FAKE, FAKE, FAKE, NULL, 4, 64, 0, 1e-6, FAKE, NULL, FAKE, ws, NULL) == -1
    assert L.moe_norm_bwd(FAKE, FAKE, FAKE, NULL, 4, 64, 0, 1e-6, FAKE, FAKE, ODD, ws, NULL) == -1
    res = L.moe_norm_residual_bwd
    # dn without w_next; neither dout nor dn; a gate without its gradient
    assert res(FAKE, FAKE, FAKE, FAKE, FAKE, NULL, 0, NULL, 4, 64, 0, 1.0, 1e-6, FAKE, FAKE, FAKE, NULL, NULL, FAKE, ws,
               NULL) == -1
    assert res(NULL, NULL, NULL, FAKE, FAKE, NULL, 0, NULL, 4, 64, 0, 1.0, 1e-6, FAKE, FAKE, FAKE, NULL, NULL, FAKE, ws,
               NULL) == -1
    assert res(FAKE, NULL, NULL, FAKE, FAKE, FAKE, 1, NULL, 4, 64, 0, 1.0, 1e-6, FAKE, FAKE, FAKE, NULL, NULL, FAKE, ws,
               NULL) == -1
