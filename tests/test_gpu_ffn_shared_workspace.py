"""One workspace for calls of the gated feed-forward block of unlike sizes, one after the other: each gives what it gives with a
workspace of its own, and leaves every arrival count at zero.

The counts lie in front of the parts of tiles that are cut along K: 8 bytes for each of 4 x 76 x 16 slices, a line of 128 bytes, and 4
bytes for each of the 256 rows of tiles that the largest number of tokens (2^22) has. A call whose tiles are cut leaves fp32 sums
behind those."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from mixture_experts_layer_histogram_gb300 import _lib as L

BF = torch.bfloat16
COUNTS = 256 + 4 * 76 * 16 * 8 + 128 + (1 << 22) // 256 * 4


def inputs(T, d, f, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s, k=1.0: (torch.randn(s, generator=g, device="cuda") * k).to(BF)  # noqa: E731
    return dict(x=r(T, d), wgu=r(2 * f, d, k=d ** -0.5), wd=r(d, f, k=f ** -0.5), dy=r(T, d))


def step(T, d, f, keep, ws, seed):
    """Forward and backward, the counts looked at after each."""
    s, e = inputs(T, d, f, seed), lambda *shape, t=BF: torch.full(shape, 3, dtype=t, device="cuda")
    ab = e(T, 2 * f, t=torch.uint8) if keep else e(T, 2 * f)
    scales = e(L.moe_act8_scale_bytes(T, 2 * f), t=torch.uint8) if keep else None
    h, y, dab, dx, dwgu, dwd = e(T, f), e(T, d), e(T, 2 * f), e(T, d), e(2 * f, d), e(d, f)
    L.moe_ffn_fwd(s["x"], s["wgu"], s["wd"], None, ab, scales, h, y, ws)
    assert L.moe_read_status(ws) == 0 and ws[:COUNTS].count_nonzero() == 0
    L.moe_ffn_bwd(s["dy"], s["x"], ab, scales, h, s["wgu"], s["wd"], None, dab, dx, dwgu, dwd, ws)
    assert L.moe_read_status(ws) == 0 and ws[:COUNTS].count_nonzero() == 0
    return y, dx, dwgu, dwd


def size(T, d, f):
    return L.moe_ffn_workspace_size(T, d, f, L.dtype_code(BF), True)


@pytest.mark.parametrize("keep", [None, "f8"])
def test_calls_of_unlike_sizes(keep):
    calls = [(389, 2048, 1024), (16384, 512, 256), (389, 2048, 1024), (234, 72, 6752), (40000, 64, 64), (5, 4096, 512), (16384, 512, 256),
             (1, 2048, 8192), (9000, 128, 2048)]
    shared = torch.zeros(max(size(*c) for c in calls), dtype=torch.uint8, device="cuda")
    for i, c in enumerate(calls):
        own = torch.zeros(size(*c), dtype=torch.uint8, device="cuda")
        for got, want in zip(step(*c, keep, shared, i), step(*c, keep, own, i)):
            assert torch.equal(got, want), c


def test_counts_after_a_graph_of_unlike_sizes():
    calls = [(389, 2048, 1024), (16384, 512, 256), (130, 8192, 2048)]
    ws = torch.zeros(max(size(*c) for c in calls), dtype=torch.uint8, device="cuda")
    want = [[t.clone() for t in step(*c, None, ws, i)] for i, c in enumerate(calls)]
    made = []
    for i, (T, d, f) in enumerate(calls):
        s, e = inputs(T, d, f, i), lambda *shape: torch.empty(shape, dtype=BF, device="cuda")
        made.append((s, e(T, 2 * f), e(T, f), e(T, d), e(T, 2 * f), e(T, d), e(2 * f, d), e(d, f)))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for s, ab, h, y, dab, dx, dwgu, dwd in made:
            L.moe_ffn_fwd(s["x"], s["wgu"], s["wd"], None, ab, None, h, y, ws)
            L.moe_ffn_bwd(s["dy"], s["x"], ab, None, h, s["wgu"], s["wd"], None, dab, dx, dwgu, dwd, ws)
    for _ in range(3):
        graph.replay()
        for (s, ab, h, y, dab, dx, dwgu, dwd), w in zip(made, want):
            assert all(torch.equal(a, b) for a, b in zip((y, dx, dwgu, dwd), w))
    assert L.moe_read_status(ws) == 0 and ws[:COUNTS].count_nonzero() == 0
