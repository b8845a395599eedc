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
