"""dv of long sums: the error that include/moe_gated.h states, for terms of either sign and of one sign.

d is summed in parts, the first of a quarter of the terms up to 1792, at least 512, the others of 512, in tensor cores that
truncate by 1.2e-9 of a sum (4.5e-9 of one of terms of one sign) for each of its terms; the parts' shares of d are their lengths'.
On top of it the float32 sum over I values has I terms of 2^-24, and the fast exp and quotient 6 units of 2^-23 as in
test_gpu_gated.py."""
import pytest
import torch

from tests import test_gpu_gated as G
from tests import helpers as Hp

pytestmark = pytest.mark.gpu

F32 = torch.float32


@pytest.fixture(scope="module")
def B():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    return Hp.lib()


@pytest.mark.parametrize("one_sign,per_term", [(False, 1.2e-9), (True, 4.5e-9)])
@pytest.mark.parametrize("H", [512, 576, 2048, 2600, 7168, 16384])
def test_dv(B, H, one_sign, per_term):
    P, I = 300, 1024
    dy, w, a = G.randn(P, H, seed=1, scale=0.1), G.randn(1, H, I, seed=2, scale=0.02), G.randn(P, 2 * I, seed=3, scale=1.5)
    if one_sign:
        dy, w = dy.abs(), w.abs()
    da, dv, ws = torch.zeros_like(a), torch.zeros(P, device="cuda"), G.workspace(B, P, H, I, 1)
    B.moe_gated_dgrad(dy, w, G.offsets_of([P]), a, da, ws, drow_w=dv)
    assert B.moe_get_device_status(ws) == B.MOE_OK
    gate, up = a.double().split(I, 1)
    terms = (dy.double() @ w[0].double()) * gate * torch.sigmoid(gate) * up
    ref = terms.sum(1)
    rounding = float(terms.abs().sum(1).norm()) * (6 * 2.0 ** -23 + I ** 0.5 * 2.0 ** -24)
    first = H if H <= 512 else max(512, 64 * min(28, H // 256 & ~1))
    length = (first * first + (H - first) * 512) / H
    assert float((dv.double() - ref).norm()) <= per_term * length * float(ref.norm()) + rounding
