"""Long sums in the gradient of weights: float32's precision, and accumulation over more rows than one part."""
import pytest
import torch

from tests import helpers as Hp
from tests.test_gpu_grouped import close, offsets_of, randn, reference, workspace

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    return Hp.lib()


@pytest.mark.parametrize("P", [512, 1024, 2048, 4096])
def test_precision_does_not_fall_with_the_length(B, P):
    """Error in norm of a float32 gradient of independent values.  A part of 256 rows is J = 16 additions of 16 rows' products,
    each truncated: half a unit of the last place on average, at most 2^-24 of the partial sum, all towards zero.  Partial sums
    grow as the root of their length, so a part's error is at most 2^-24 sum_j sqrt(j / J) < 2^-24 (2/3 J + 1) of it, and the
    parts' errors are independent.  Each of the n = P / 256 additions of a part rounds to nearest, at most 2^-24 of the sum so
    far, independently: 2^-24 sqrt(n / 2)."""
    N, K = 256, 256
    dy, x, dw = randn(P, N, seed=7), randn(P, K, seed=8), torch.empty(1, N, K, device="cuda")
    B.moe_grouped_wgrad(dy, x, offsets_of([P]), dw, workspace(B, P, N, K, 1))
    ref = dy.double().T @ x.double()
    bound = 2.0 ** -24 * (2 / 3 * 16 + 1 + (P / 256 / 2) ** 0.5)
    assert float((dw[0].double() - ref).norm() / ref.norm()) <= bound


@pytest.mark.parametrize("counts", [[1500, 0, 257, 4133], [5000], [256, 255, 512, 513, 1]])
def test_accumulation_over_parts(B, counts):
    E, P, N, K = len(counts), sum(counts), 136, 328
    dy, x = randn(P, N, seed=5), randn(P, K, seed=6)
    g = torch.Generator(device="cuda").manual_seed(1)
    base = torch.randn(E, N, K, generator=g, device="cuda")
    dw, ws = base.clone(), workspace(B, P, N, K, E)
    for times in (1, 2):
        B.moe_grouped_wgrad(dy, x, offsets_of(counts), dw, ws, accumulate=True)
        assert B.moe_get_device_status(ws) == B.MOE_OK
        for e, (_, _, ref, mag, terms) in enumerate(reference("wgrad", counts, dy, x)):
            close(dw[e], base[e].double() + times * ref, base[e].double().abs() + times * mag, terms + times)
            if counts[e] == 0:
                assert torch.equal(dw[e], base[e])
