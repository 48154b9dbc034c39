"""The MXFP4 FFN on offsets that contradict tile_offsets or the buffers: the experts concerned are skipped and reported,
the others are computed, and nothing is written outside the buffers (which lie between guard rows here). Both sets of
kernels: few rows per expert, and many."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from mixture_experts_layer_histogram_gb300 import Fp4Weights, fp4_quantize
    from mixture_experts_layer_histogram_gb300 import _lib as L

D = F = 256
R = 512
GUARD = 256
GOOD = {2: ([0, 2, 4], [0, 200, 330]), 8: ([0, 1, 1, 2, 2, 3, 3, 3, 4], [0, 5, 5, 69, 69, 79, 79, 79, 207])}
# E: [(tile_offsets, offsets, experts that stay right)]
BAD = {
    2: [([0, 1, 2], [0, 300, 330], []),                      # 300 rows in one group; expert 1 then starts elsewhere
        ([0, 2, 4], [0, 200, 600], [0]),                     # 400 rows in two groups
        ([0, 2, 9], [0, 200, 330], [0]),                     # a group that ends past the buffers
        ([-3, 2, 4], [0, 200, 330], [1]),                    # one that starts before them
        ([0, 2, 1], [0, 200, 330], [0]),                     # groups that run backwards
        ([0, 2, 4], [0, 200, 150], [0])],                    # a negative count
    8: [([0, 1, 1, 2, 2, 3, 3, 3, 90], GOOD[8][1], [0, 2, 4]),
        ([0, 1, 1, 2, 2, 3, 3, 3, 4], [0, 5, 5, 200, 200, 210, 210, 210, 338], [0, 4, 7]),
        ([0, 1, 1, 2, 2, 3, 3, 3, 4], [0, 5, 5, -60, -60, -50, -50, -50, 78], [0, 4, 7]),
        ([0, 1, -7, 2, 2, 3, 3, 3, 4], GOOD[8][1], [0, 4, 7]),
        ([1 << 24, 1, 1, 2, 2, 3, 3, 3, 4], GOOD[8][1], [2, 4, 7])],
}
CASES = [(E, i) for E in BAD for i in range(len(BAD[E]))]


def guarded(cols, dtype, fill):
    t = torch.full((GUARD + R + GUARD, cols), fill, dtype=dtype, device="cuda")
    return t, t[GUARD:GUARD + R]


def run(E, toff, off, x, w):
    h, hv = guarded(F // 2, torch.uint8, 0xEE)
    s, sv = guarded(F // 32, torch.uint8, 0xEE)              # scales: four bytes per row and 128 features
    y, yv = guarded(D, torch.bfloat16, 7.0)
    ws = torch.zeros(L.moe_grouped_ffn_workspace_size(E, D, F, R, L.MOE_BF16, False), dtype=torch.uint8, device="cuda")
    L.moe_grouped_ffn_fwd_fp4(*x, w.gate_up, w.gate_up_scales, w.down, w.down_scales,
                              torch.tensor(toff, dtype=torch.int32, device="cuda"),
                              torch.tensor(off, dtype=torch.int32, device="cuda"), hv, sv.reshape(-1), yv, ws)
    status = L.moe_read_status(ws)
    for t, fill in ((h, 0xEE), (s, 0xEE), (y, 7.0)):
        assert t[:GUARD].eq(fill).all() and t[GUARD + R:].eq(fill).all()
    return status, yv


def operands(E):
    g = torch.Generator(device="cuda").manual_seed(E)
    x = fp4_quantize(torch.randn(R, D, generator=g, device="cuda"))
    w = Fp4Weights.quantize(torch.randn(E, 2 * F, D, generator=g, device="cuda") * 0.05,
                            torch.randn(E, D, F, generator=g, device="cuda") * 0.05)
    return x, w


@pytest.mark.parametrize("E,case", CASES)
def test_contradicting_offsets(E, case):
    x, w = operands(E)
    good = GOOD[E]
    status, want = run(E, *good, x, w)
    assert status == 0
    toff, off, right = BAD[E][case]
    status, y = run(E, toff, off, x, w)
    assert status == -6
    for e in right:
        lo, n = good[0][e] * 128, good[1][e + 1] - good[1][e]
        if off[e + 1] - off[e] == n and toff[e] == good[0][e]:
            assert n > 0 and torch.equal(y[lo:lo + n], want[lo:lo + n]), e
        else:
            raise AssertionError("the case's list of right experts is wrong")


@pytest.mark.parametrize("counts,toff", [([-1000, 3], [0, 1]), ([5, 3], [-2, 0]), ([5, 3], [0, -1])])
def test_permutation_with_groups_before_the_buffers(counts, toff):
    """Padding rows that would lie before the buffers are not written."""
    E, k, T = 2, 1, 1
    rows = L.moe_grouped_rows_max(T, k, E)
    buf = torch.full((2048 + rows, 128 // 2), 0xEE, dtype=torch.uint8, device="cuda")
    scales = torch.full((2048 + rows, 4), 0xEE, dtype=torch.uint8, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    L.moe_permute_fp4(torch.ones(T, 128, device="cuda"), k, E, torch.tensor([-1], **i32), torch.tensor(counts, **i32),
                      torch.tensor(toff + [toff[1] + 1], **i32), buf[2048:], scales[2048:].reshape(-1))
    torch.cuda.synchronize()
    assert buf[:2048].eq(0xEE).all() and scales[:2048].eq(0xEE).all()
