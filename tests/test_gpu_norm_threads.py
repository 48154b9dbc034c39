"""Block norms called from two host threads at once, at widths that need different amounts of shared memory: every
call is valid, so every call succeeds and gives what it gives alone."""
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from mixture_experts_layer_histogram_gb300 import BlockNorms
    from mixture_experts_layer_histogram_gb300 import _lib as L


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_two_threads_two_widths(dtype):
    """2048 and 4096 bf16 (1024 and 2048 fp32) channels run the same instantiation of the backward, with rings of 61 and 123
    KB. The C entry point is called straight, so that the two threads are inside it at the same time."""
    T, rounds = 4, 20000
    errors, start = [], threading.Barrier(2)
    code = L.dtype_code(dtype)

    def work(d, args, got, want, stream):
        try:
            fn = L.lib().moe_norm_residual_bwd
            start.wait()
            for i in range(rounds):
                rc = fn(*args)
                assert rc == 0, (d, i, rc)
            stream.synchronize()
            for a, b in zip(got, want):
                assert torch.equal(a, b), d
        except Exception as e:   # the main thread reports it
            errors.append(e)

    threads, keep = [], []
    for d in (2048, 4096) if dtype == torch.bfloat16 else (1024, 2048):
        g = torch.Generator(device="cuda").manual_seed(d)
        dout, dn, out, y = (torch.randn(T, d, generator=g, device="cuda").to(dtype) for _ in range(4))
        w = torch.randn(d, generator=g, device="cuda").to(dtype)
        norms = BlockNorms(T, d, dtype)
        res = norms.post_backward(dout, dn, out, y, w, w_next=w)
        want = [v.clone() for v in res.values()]
        for v in res.values():
            v.zero_()
        stream = torch.cuda.Stream()
        n = norms
        args = (dout.data_ptr(), dn.data_ptr(), out.data_ptr(), y.data_ptr(), w.data_ptr(), None, 0, w.data_ptr(), T, d, code,
                1.0, 1e-6, n.dx.data_ptr(), n.dy.data_ptr(), n.dw_post.data_ptr(), None, n.dw_next.data_ptr(),
                n.ws.data_ptr(), n.ws.numel(), stream.cuda_stream)
        keep.append((dout, dn, out, y, w, norms, stream))
        threads.append(threading.Thread(target=work, args=(d, args, list(res.values()), want, stream)))
    torch.cuda.synchronize()
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors, errors
