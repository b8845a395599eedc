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
