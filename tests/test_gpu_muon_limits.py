"""The ends of what include/moe_muon.h allows: polynomials near the largest factor, and matrices of low rank.

Tolerances: test_gpu_muon.py's, against the definition with the kernels' roundings; and the header's figures for matrices of
rank 1, 4 and 16, two digits each, so half a hundredth above them."""
import pytest
import torch

from tests import test_gpu_muon as T
from tests import helpers as Hp

pytestmark = pytest.mark.gpu

F32 = torch.float32


@pytest.fixture(scope="module")
def B():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    return Hp.lib()


@pytest.mark.parametrize("how", [dict(coefficients=(15.5, -14.0, 1.0)), dict(coefficients=(-15.5, 14.0, -1.0)),
                                 dict(coefficients=(1.0, 14.5, 0.0)), dict(coefficients=(1.0, 56.0, -56.0))])
@pytest.mark.parametrize("shape", [(2, 72, 136), (2, 136, 72), (2, 200, 264)])
def test_largest_factors(B, shape, how):
    x = T.randn(*shape, seed=5, scale=1e-3, dtype=F32)
    T.check(T.ortho(B, x, F32, steps=1, **how), x, steps=1, **how)
    assert bool((T.ortho(B, torch.zeros_like(x), **how) == 0).all())


@pytest.mark.parametrize("rank,most", [(1, 0.15), (4, 0.08), (16, 0.05)])
@pytest.mark.parametrize("shape", [(64, 200), (128, 384), (2000, 128), (256, 640), (520, 264), (1024, 2048)])
def test_matrices_of_low_rank(B, shape, rank, most):
    """As the gradient of an expert with few tokens: the polynomial enlarges what the roundings leave in the directions that
    the matrix lacks."""
    N, K = shape
    x = (T.randn(N, rank, seed=1, dtype=F32) @ T.randn(rank, K, seed=2, dtype=F32))[None]
    got = T.ortho(B, x, F32)
    T.check(got, x)
    assert T.error(got[0], T.orthogonal(x[0])) <= most + 0.005


@pytest.mark.parametrize("shape", [(30, 3383), (300, 1000), (1000, 300), (31, 4100), (1024, 2048), (2050, 700), (129, 900), (136, 264)])
def test_products_keep_their_diagonals(B, shape):
    """As test_gpu_muon.py's test of small matrices, for those that go through the products: the roundings' draw plays no part but
    for 1.5 times, and a sum's terms add 2^-23 each at most."""
    x = T.randn(3, *shape, seed=sum(shape), scale=1e-3, dtype=F32)
    for o, m in list(zip(T.ortho(B, x, F32), x))[:2]:
        emulated = T.kept_diagonals(m)
        ref = T.orthogonal(m)
        bound = 1.5 * T.error(emulated.T if shape[0] > shape[1] else emulated, ref) + max(shape) * 2.0 ** -23
        assert T.error(o, ref) <= bound, (T.error(o, ref), bound)
