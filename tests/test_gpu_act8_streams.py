"""Activations to 8 bits and back on another stream than the current one, whose freed memory is still being written."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from mixture_experts_layer_histogram_gb300 import act8_dequantize, act8_quantize

R, K = 8192, 4096          # (tensors of more than 10 MB have memory blocks of their own size)


def busy_memory(dtype, shape):
    """The address of a block of the current stream's memory, the only one of its size that is free, while a fill of it waits behind
    some milliseconds of products."""
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    m = torch.randn(2048, 2048, device="cuda")
    t = torch.empty(shape, dtype=dtype, device="cuda")
    torch.cuda.synchronize()
    for _ in range(100):
        torch.mm(m, m)
    t.fill_(77)
    return t.data_ptr()


@pytest.mark.parametrize("back", [False, True])
def test_results_have_memory_of_their_stream(back):
    torch.cuda.empty_cache()
    x = torch.empty(R, K, dtype=torch.bfloat16, device="cuda").normal_()    # (no temporaries: every block is as large as its tensor)
    codes, scales = act8_quantize(x)
    values = act8_dequantize(codes, scales)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    if back:
        busy = busy_memory(torch.bfloat16, (R, K))
        got = [act8_dequantize(codes, scales, stream=side)]
        want = [values]
    else:
        busy = busy_memory(torch.uint8, (R, K))
        got, want = act8_quantize(x, stream=side), [codes, scales]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and got[0].data_ptr() != busy


def test_into_out():
    x = torch.randn(8, 96, device="cuda").bfloat16()
    codes, scales = act8_quantize(x)
    side, out = torch.cuda.Stream(), torch.empty_like(x)
    torch.cuda.synchronize()
    assert act8_dequantize(codes, scales, out=out, stream=side) is out
    torch.cuda.synchronize()
    assert torch.equal(out, act8_dequantize(codes, scales))
