"""Stacks that the orthogonalisation and Muon refuse for their number of tiles (without a GPU).

A refused step enqueues nothing: on a machine without a GPU the first launch would answer MOE_ERR_CUDA, and with one it would
have moved the momentum."""
import pytest

from tests import helpers as Hp
from tests.test_muon_abi import ORTHO, STEP, call

# 4098 tiles a matrix and iteration: 1.7e10 in all, more than an item's number holds
STACK = dict(E=65535, N=1, K=(1 << 20) - 8, workspace_bytes=1 << 60)


@pytest.mark.parametrize("name,kind,base", [("moe_muon_step", "MoeMuonArgs", STEP), ("moe_orthogonalize", "MoeOrthogonalizeArgs", ORTHO)])
@pytest.mark.parametrize("change", [{}, dict(N=(1 << 20) - 8, K=1)])
def test_a_stack_of_too_many_tiles_is_refused_before_the_first_launch(name, kind, base, change):
    B = Hp.lib()
    got = call(B, name, getattr(B, kind), base, {**STACK, **change, "ns": dict(steps=64)})
    assert got == B.MOE_ERR_UNSUPPORTED_SHAPE


@pytest.mark.parametrize("a,b,c,ok", [
    (20.0, -4.775, 2.0315, False), (-16.0, 1.0, 0.0, False), (1.0, 15.5, 0.0, False), (0.0, 8.0, 8.0, False),       # at 0, at 1
    (1.0, 61.0, -60.0, False), (-1.0, -61.0, 60.0, False),                                # at 1/2, with 2 and -2 at the ends
    (15.5, -14.0, 1.0, True), (-15.5, 14.0, -1.0, True), (1.0, 14.5, 0.0, True), (1.0, 56.0, -56.0, True), (0.0, 0.0, 0.0, True)])
@pytest.mark.parametrize("name,kind,base", [("moe_muon_step", "MoeMuonArgs", STEP), ("moe_orthogonalize", "MoeOrthogonalizeArgs", ORTHO)])
def test_polynomials_whose_factor_passes_fp16_are_refused(name, kind, base, a, b, c, ok):
    """a + b t + c t^2 over the Gram matrix's eigenvalues, 0 .. 1: FP16 with a scale of 2^12 ends at 15.99."""
    B = Hp.lib()
    change = dict(E=0, workspace=0, workspace_bytes=0, ns=dict(a=a, b=b, c=c))          # no matrices: nothing but the checks
    assert call(B, name, getattr(B, kind), base, change) == (B.MOE_OK if ok else B.MOE_ERR_INVALID_ARG)
