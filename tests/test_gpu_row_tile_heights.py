"""Each height of a tile of rows (64, 128, 256) for each product that chooses one: plain and gated, both directions, with
several experts, some without rows.

``height`` is the kernels' rule for this GPU's number of SMs, so that a case that no longer reaches its height fails.  The
tolerances are those of test_gpu_grouped.py and test_gpu_gated.py."""
import pytest
import torch

from tests import test_gpu_gated as G
from tests import test_gpu_grouped as P0
from tests import helpers as Hp

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
R = 328                          # length of the gated products' sums

# counts, columns of the product, length of its sums, height
PLAIN = [([300, 0, 40, 130], 400, 584, 64), ([70, 64, 65, 129], 136, 328, 64), ([690, 0, 450, 33, 40], 1000, 584, 128),
         ([0, 1100, 80], 904, 1032, 128), ([20] * 12, 400, 584, 256), ([900, 0, 800], 1400, 584, 256), ([2100, 640], 264, 520, 128),
         ([96, 20, 0, 90], 400, 328, 256)]
# counts, columns (gate and up rows forward), height
GATED = [([300, 0, 40, 130], 400, 64), ([0, 65, 128, 1, 200], 528, 64), ([700, 0, 500, 33], 1392, 128),
         ([260, 130, 0, 5, 700], 1200, 128), ([400, 0, 300, 20], 4000, 256), ([40] * 9, 2560, 256)]


@pytest.fixture(scope="module")
def B():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    return Hp.lib()


def up(a, b):
    return -(-a // b)


def height(counts, columns, gated, pairs):
    """csrc/grouped_kernel.cuh: most_row_items() says which launches look, log_rows() what they choose."""
    P, E, mt = sum(counts), len(counts), up(columns, 256)
    if P <= 64 or up(P, 128) * mt > pairs or max(counts) <= (64 if gated else 96):
        return 256
    pairs = min(pairs, min(P, P // 64 + E) * mt)
    return next((t for t in (64, 128) if sum(up(c, t) for c in counts) * mt <= pairs), 256)


def expect(counts, columns, gated, want):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    for pairs in (sms // 2, sms // 2 - 2):                  # not at the edge
        assert height(counts, columns, gated, pairs) == want


@pytest.mark.parametrize("counts,columns,sums,want", PLAIN)
@pytest.mark.parametrize("op", ["forward", "dgrad"])
def test_products(B, op, counts, columns, sums, want):
    expect(counts, columns, False, want)
    E, P = len(counts), sum(counts)
    N, K = (columns, sums) if op == "forward" else (sums, columns)
    x, w = P0.randn(P, sums, seed=1), P0.randn(E, N, K, seed=2, scale=0.1)
    out, ws = torch.full((P + 1, columns), 3.0, dtype=BF16, device="cuda"), P0.workspace(B, P, N, K, E)
    (B.moe_grouped_forward if op == "forward" else B.moe_grouped_dgrad)(x, w, P0.offsets_of(counts), out[:P], ws)
    assert B.moe_get_device_status(ws) == B.MOE_OK and bool((out[P] == 3).all())
    for a, b, ref, mag, terms in P0.reference(op, counts, x, w):
        P0.close(out[a:b], ref, mag, terms)


@pytest.mark.parametrize("case", range(len(GATED)))
def test_gated(B, case):
    counts, columns, want = GATED[case]
    expect(counts, columns, True, want)
    E, P, I = len(counts), sum(counts), columns // 2
    row_w = G.randn(P, seed=3, dtype=F32)
    x, w = G.randn(P, R, seed=1), G.randn(E, 2 * I, R, seed=2, scale=1.5 * R ** -0.5)
    h, a = torch.full((P + 1, I), 3.0, dtype=BF16, device="cuda"), torch.full((P + 1, 2 * I), 3.0, dtype=BF16, device="cuda")
    ws = G.workspace(B, P, R, I, E)
    B.moe_gated_forward(x, w, G.offsets_of(counts), h[:P], ws, a=a[:P], row_w=row_w, activation=case % 2)
    assert B.moe_get_device_status(ws) == B.MOE_OK and bool((h[P] == 3).all()) and bool((a[P] == 3).all())
    G.check_forward(h, a, x, w, row_w, counts, case % 2)


@pytest.mark.parametrize("case", range(len(GATED)))
def test_the_way_back(B, case):
    counts, I, want = GATED[case]
    expect(counts, I, True, want)
    E, P = len(counts), sum(counts)
    dy, w, a = G.randn(P, R, seed=4), G.randn(E, R, I, seed=5, scale=R ** -0.5), G.randn(P, 2 * I, seed=6)
    row_w = G.randn(P, seed=3, dtype=F32)
    out = {"da": torch.full((P + 1, 2 * I), 3.0, dtype=BF16, device="cuda"), "h": torch.full((P + 1, I), 3.0, dtype=BF16, device="cuda"),
           "drow_w": torch.full((P + 1,), 3.0, device="cuda")}
    ws = G.workspace(B, P, R, I, E)
    B.moe_gated_dgrad(dy, w, G.offsets_of(counts), a, out["da"][:P], ws, h=out["h"][:P], row_w=row_w, drow_w=out["drow_w"][:P],
                      activation=case % 2)
    assert B.moe_get_device_status(ws) == B.MOE_OK and all(bool((t[P] == 3).all()) for t in out.values())
    G.check_back(out, dy, w, a, row_w, counts, case % 2)
