"""Tiles of fewer rows, where a launch has few: the products grouped by expert and the gated block on both sides of the
choice.

The tolerances are those of test_gpu_grouped.py and test_gpu_gated.py: a tile's rows do not change a value's sum.  For the
same reason an expert's rows have the same bits whatever tiles they fall in.
"""
import pytest
import torch

from tests import test_gpu_gated as G
from tests import test_gpu_grouped as P0
from tests import helpers as Hp

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32

# counts, I, H.  Of 152 SMs, 76 pairs: the first four are cut into tiles of 64 rows, the next three of 128, the last four
# not at all, forward and gated (2 I columns); the gradients (I, or H) also.
SIZES = [
    ([300], 136, 72), ([65], 24, 200), ([0, 320, 0, 64, 63, 1, 129], 128, 136), ([1000, 577], 72, 264),
    ([1024], 1024, 1096), ([700, 0, 500, 33], 1104, 1032), ([1800], 520, 520),
    ([320, 576, 257, 1, 64], 2568, 2600), ([1025, 0, 300], 2048, 2056), ([264], 5000, 5128), ([130, 700, 0, 321, 640], 1544, 1800),
]


@pytest.fixture(scope="module")
def B():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    return Hp.lib()


@pytest.mark.parametrize("case", range(len(SIZES)))
@pytest.mark.parametrize("op", ["forward", "dgrad"])
def test_products(B, op, case):
    counts, I, H = SIZES[case]
    E, P = len(counts), sum(counts)
    R, M = (H, I) if op == "forward" else (I, H)
    x, w = P0.randn(P, R, seed=1), P0.randn(E, I, H, seed=2, scale=0.1)
    out, ws = torch.full((P + 1, M), 3.0, dtype=BF16, device="cuda"), P0.workspace(B, P, I, H, E)
    (B.moe_grouped_forward if op == "forward" else B.moe_grouped_dgrad)(x, w, P0.offsets_of(counts), out[:P], ws)
    assert B.moe_get_device_status(ws) == B.MOE_OK and bool((out[P] == 3).all())
    for a, b, ref, mag, terms in P0.reference(op, counts, x, w):
        P0.close(out[a:b], ref, mag, terms)


@pytest.mark.parametrize("case", range(len(SIZES)))
def test_gated(B, case):
    counts, I, H = SIZES[case]
    E, P, first = len(counts), sum(counts), case % 3
    n = P + 2 * first
    own = slice(first, first + P)
    row_w = G.randn(n, seed=3, dtype=F32)
    x, w = G.randn(n, H, seed=1), G.randn(E, 2 * I, H, seed=2, scale=1.5 * H ** -0.5)
    h, a = torch.full((n, I), 3.0, dtype=BF16, device="cuda"), torch.full((n, 2 * I), 3.0, dtype=BF16, device="cuda")
    ws = G.workspace(B, n, H, I, E)
    B.moe_gated_forward(x, w, G.offsets_of(counts, first), h, ws, a=a, row_w=row_w, activation=case % 2)
    assert B.moe_get_device_status(ws) == B.MOE_OK
    G.check_forward(h, a, x, w, row_w, counts, case % 2, first)
    dy, down = G.randn(n, H, seed=4), G.randn(E, H, I, seed=5, scale=H ** -0.5)
    out = {"da": torch.full((n, 2 * I), 3.0, dtype=BF16, device="cuda"), "h": torch.full((n, I), 3.0, dtype=BF16, device="cuda"),
           "drow_w": torch.full((n,), 3.0, device="cuda")}
    B.moe_gated_dgrad(dy, down, G.offsets_of(counts, first), a, out["da"], ws, h=out["h"], row_w=row_w, drow_w=out["drow_w"],
                      activation=case % 2)
    assert B.moe_get_device_status(ws) == B.MOE_OK
    G.check_back(out, dy, down, a, row_w, counts, case % 2, first)
    for t in (h, a, *out.values()):
        t[own] = 3.0
        assert bool((t == 3).all())


@pytest.mark.parametrize("counts", [[300], [65, 0, 320, 129], [700, 64]])
def test_bits_do_not_depend_on_the_tiles(B, counts):
    """One more expert of many rows, and the others' tiles are as large as they get."""
    I, H, many = 136, 264, 12000
    E, P = len(counts), sum(counts)
    n, row_w = P + many, G.randn(P + many, seed=3, dtype=F32)
    x, w, down = G.randn(n, H, seed=1), G.randn(E + 1, 2 * I, H, seed=2, scale=0.1), G.randn(E + 1, H, I, seed=5, scale=0.1)
    kept = G.randn(n, 2 * I, seed=6)

    def run(k, rows):
        offsets = G.offsets_of([*counts, many][:k])
        new = lambda *shape, dtype=BF16: torch.zeros(*shape, dtype=dtype, device="cuda")       # noqa: E731
        out = {"h": new(rows, I), "a": new(rows, 2 * I), "da": new(rows, 2 * I), "drow_w": new(rows, dtype=F32),
               "y": new(rows, 2 * I), "dx": new(rows, H)}
        ws, wg = G.workspace(B, rows, H, I, k), P0.workspace(B, rows, 2 * I, H, k)
        B.moe_gated_forward(x[:rows], w[:k], offsets, out["h"], ws, a=out["a"], row_w=row_w[:rows])
        B.moe_gated_dgrad(x[:rows], down[:k], offsets, kept[:rows], out["da"], ws, row_w=row_w[:rows], drow_w=out["drow_w"])
        B.moe_grouped_forward(x[:rows], w[:k], offsets, out["y"], wg)
        B.moe_grouped_dgrad(kept[:rows], w[:k], offsets, out["dx"], wg)
        assert B.moe_get_device_status(ws) == B.MOE_OK and B.moe_get_device_status(wg) == B.MOE_OK
        return out

    few, all_ = run(E, P), run(E + 1, n)
    for k, t in few.items():
        assert torch.equal(t, all_[k][:P]), k
