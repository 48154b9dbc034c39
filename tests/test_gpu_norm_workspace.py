"""The norms' backward keeps to its workspace: bytes behind it are not written, for each number of inputs and widths around
which the ring of rows loses a stage (fewer stages leave room for more blocks, each with a partial row)."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from mixture_experts_layer_histogram_gb300 import _lib as L


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("d", [33, 1537, 2048, 3413, 3414, 4267, 5120, 5124, 5376, 6827, 8191, 8192])
def test_nothing_behind_the_workspace(d, dtype):
    T = 2500
    size = L.moe_norm_bwd_workspace_size(T, d, L.dtype_code(dtype))
    g = torch.Generator(device="cuda").manual_seed(d)
    x, y, dn, dout, gate = (torch.randn(T, d, generator=g, device="cuda").to(dtype) for _ in range(5))
    w = torch.randn(d, generator=g, device="cuda").to(dtype)
    dx, dy, dgate = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x)
    dw, dwn = torch.empty_like(w), torch.empty_like(w)
    buf = torch.full((size + (1 << 24),), 0xA5, dtype=torch.uint8, device="cuda")
    ws = buf[:size]
    for dx_in in (None, dout):
        L.moe_norm_bwd(dn, x, w, dx_in, dx, dw, ws)
    for do in (None, dout):
        for gt, dg in ((None, None), (gate, dgate)):
            L.moe_norm_residual_bwd(do, dn, x, y, w, gt, w, dx, dy, dw, dg, dwn, ws)
            if do is not None:
                L.moe_norm_residual_bwd(do, None, None, y, w, gt, None, dx, dy, dw, dg, None, ws)
    torch.cuda.synchronize()
    assert buf[size:].eq(0xA5).all()
