"""The norms' gradients at the edges of float32's range, and with infinities where a formula does not read them.

Tolerance as in test_gpu_norm.py: (H + T + 64) * 2^-23 of the sum of the terms' magnitudes, and the output's rounding.
"""
import pytest
import torch

from tests import helpers as Hp
from tests.test_gpu_norm import Case, backward64, close

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def M():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    Hp.lib()
    import moe_expert_layer_counting_gb300
    return moe_expert_layer_counting_gb300


@pytest.mark.parametrize("gate", [None, "token", "channel", "full"])
@pytest.mark.parametrize("H,xt", [(1024, BF16), (1024, F32), (8200, BF16), (8200, F32)])
@pytest.mark.parametrize("y_exp,b_exp", [(-46, 0), (50, 0), (0, -46), (0, 50), (-46, 50), (50, -46)])
def test_gradients_of_rows_far_from_one(M, y_exp, b_exp, H, xt, gate):
    """Rows of 2^-46 or 2^50 times the usual magnitude, without eps: squares, their sums and the results are well inside
    float32, the cube of a norm's reciprocal is not (2^138, 2^-150).  No dy, so that the norm's gradient is all of dx."""
    c = Case(40, H, xt, gate=gate, sigmoid=gate == "full", eps=0.0)
    y = c.x * 2.0 ** y_exp
    c.b, c.dy = c.b * 2.0 ** b_exp, None
    got, want = c.module(M).backward(y, c.b, c.gate, None, c.dn), backward64(c, y)
    assert {k for k, v in got.items() if v is not None} == set(want)
    for k in want:
        close(k, got[k].reshape(want[k][0].shape), want[k], H, c.T)


@pytest.mark.parametrize("gate", [None, "token", "channel", "full"])
@pytest.mark.parametrize("H,xt", [(264, BF16), (264, F32), (8200, BF16)])
def test_gradient_of_b_without_a_norm_does_not_read_b(M, H, xt, gate):
    """u = b: db = g d, finite where b is not; the gate's gradient d b is not finite there."""
    c = Case(30, H, xt, gate=gate, post=False)
    y, want = c.x.clone(), backward64(c, c.x)
    c.b[7, 5], c.b[11, H - 1] = float("inf"), float("nan")
    got = c.module(M).backward(y, c.b, c.gate, c.dy, c.dn)
    for k in ("dx", "db", "dw_pre"):
        close(k, got[k], want[k], H, c.T)
    if gate == "token":
        fine = got["dgate"][:, 0].isfinite()
        assert not bool(fine[7]) and not bool(fine[11]) and int(fine.sum()) == 28


@pytest.mark.parametrize("kind,gt", [("token", BF16), ("token", F32), ("channel", BF16), ("channel", F32)])
def test_gates_gradients_aligned_as_their_elements(M, kind, gt):
    """A token gate and the gradient of a token's or channel's gate may start at any element."""
    B = M.binding
    c = Case(33, 264, gate=kind, gt=gt, sigmoid=True)
    held = torch.full((c.gate.numel() + 2,), 7.0, dtype=gt, device="cuda")
    dgate = held[1:-1].view(c.gate.shape)
    if kind == "token":
        c.gate = torch.cat([c.gate[:1], c.gate])[1:]
    ws = torch.empty(B.moe_norm_workspace_size(c.T, c.H), dtype=torch.uint8, device="cuda")
    B.moe_norm_backward(c.x, c.b, c.gate, c.w_post, c.w_pre, c.dy, c.dn, ws, dgate=dgate, residual_scale=c.scale, eps=c.eps,
                        gate_sigmoid=True)
    close("dgate", dgate, backward64(c, c.x)["dgate"], c.H, c.T)
    assert float(held[0]) == float(held[-1]) == 7.0
