"""dv of long sums: the error that include/moe_gated.h states, for terms of either sign and of one sign; and the
sums in parts at ragged sizes, in place, with NaN and with a wait that runs out.

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


COUNTS, I, H = [300, 0, 33, 257, 320, 1, 576], 200, 1096          # sums in parts, experts around one and two tiles


def problem(B):
    P, E = sum(COUNTS), len(COUNTS)
    t = {"dy": G.randn(P + 8, H, seed=1), "w": G.randn(E, H, I, seed=2, scale=H ** -0.5), "a": G.randn(P + 8, 2 * I, seed=3),
         "row_w": G.randn(P + 8, seed=4, dtype=F32), "ws": G.workspace(B, P + 8, H, I, E), "offsets": G.offsets_of(COUNTS, 4)}
    t["out"] = {"da": torch.full_like(t["a"], 3.0), "h": torch.full((P + 8, I), 3.0, dtype=torch.bfloat16, device="cuda"),
                "drow_w": torch.full((P + 8,), 3.0, device="cuda")}
    return t


def back(B, t, da=None):
    B.moe_gated_dgrad(t["dy"], t["w"], t["offsets"], t["a"], t["out"]["da"] if da is None else da, t["ws"], h=t["out"]["h"],
                      row_w=t["row_w"], drow_w=t["out"]["drow_w"])
    return B.moe_get_device_status(t["ws"])


def test_parts_in_place_and_again(B):
    t = problem(B)
    assert back(B, t) == B.MOE_OK
    G.check_back(t["out"], t["dy"], t["w"], t["a"], t["row_w"], COUNTS, 0, 4)
    first = {k: v.clone() for k, v in t["out"].items()}
    own = slice(4, 4 + sum(COUNTS))
    assert all(bool((v[:4] == 3).all()) and bool((v[own.stop:] == 3).all()) for v in first.values())
    before = t["a"].clone()
    assert back(B, t, da=t["a"]) == B.MOE_OK                         # over a itself
    assert torch.equal(t["a"][own], first["da"][own]) and torch.equal(t["a"][:4], before[:4]) and torch.equal(t["a"][own.stop:], before[own.stop:])
    assert torch.equal(t["out"]["drow_w"], first["drow_w"]) and torch.equal(t["out"]["h"], first["h"])


def test_parts_keep_nan_in_their_rows(B):
    t = problem(B)
    assert back(B, t) == B.MOE_OK
    clean = {k: v.clone() for k, v in t["out"].items()}
    rows = torch.tensor([4, 4 + 299, 4 + 300, 4 + 340, 4 + 700, 4 + sum(COUNTS) - 1], device="cuda")
    t["dy"][rows, 77] = float("nan")
    t["dy"][:4] = float("inf")                                       # rows of no expert
    assert back(B, t) == B.MOE_OK
    others = torch.ones(t["dy"].shape[0], dtype=torch.bool, device="cuda")
    others[rows] = False
    assert all(torch.equal(clean[k][others], v[others]) for k, v in t["out"].items())
    assert bool(t["out"]["drow_w"][rows].isnan().all()) and torch.equal(t["out"]["h"], clean["h"])


def test_a_wait_that_runs_out_between_parts_is_reported(B, monkeypatch):
    t = problem(B)
    monkeypatch.setenv("MOE_MXQ_DEBUG_INJECT_WAIT", "1")
    assert back(B, t) == B.MOE_ERR_TIMEOUT and bool((t["out"]["drow_w"] == 3).all())
    monkeypatch.delenv("MOE_MXQ_DEBUG_INJECT_WAIT")
    assert back(B, t) == B.MOE_OK
    G.check_back(t["out"], t["dy"], t["w"], t["a"], t["row_w"], COUNTS, 0, 4)
