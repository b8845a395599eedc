"""A wait of the norms that gives up, without a fault: the debug hook makes the first thread wait for what never comes
(~10 ms), and so others wait for what it does not bring (~1 s).  The call ends, its status says so, what was not computed is NaN, and the next call is right."""
import time

import pytest
import torch

from tests import helpers as Hp
from tests.test_gpu_norm import Case, backward64, close, forward64

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def M():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    Hp.lib()
    import moe_expert_layer_counting_gb300
    return moe_expert_layer_counting_gb300


CASES = [dict(T=1, H=64), dict(T=3000, H=512, gate="token"), dict(T=700, H=4096, xt=F32, gate="channel"),
         dict(T=700, H=7168, gate="full"), dict(T=400, H=8200, gate="channel"), dict(T=300, H=16384, xt=F32, post=False),
         dict(T=600, H=1024, post=False, gate="channel"), dict(T=600, H=1024, layer=False), dict(T=400, H=9000, layer=False)]


@pytest.mark.parametrize("how", CASES)
def test_forward(M, monkeypatch, how):
    B, c = M.binding, Case(**how)
    m, want = c.module(M), forward64(c)
    monkeypatch.setenv("MOE_MXQ_DEBUG_INJECT_WAIT", "1")
    t0 = time.perf_counter()
    y, n = m.forward(c.x, c.b, c.gate)
    assert m.device_status() == B.MOE_ERR_TIMEOUT
    assert time.perf_counter() - t0 < 5.0
    # the first row is lost; every row is NaN in n or as it should be, its y too but for the lost columns of a layer without
    # a norm of its own
    bad = n.isnan().all(1)
    assert bool(bad[0]) and int(bad.sum()) <= -(-c.T // 50)
    close("n", n[~bad], tuple(v[~bad] for v in want["n"]), c.H, 0)
    if c.b is not None:
        off = y.isnan()
        assert not bool(off[~bad].any()) and bool(off[bad].any(1).all())
        if c.w_post is not None:
            assert bool(off[bad].all())
        close("y", torch.where(off, 0, y), tuple(torch.where(off, 0.0, v) for v in want["y"]), c.H, 0)
    monkeypatch.delenv("MOE_MXQ_DEBUG_INJECT_WAIT")
    y, n = m.forward(c.x, c.b, c.gate)
    assert m.device_status() == B.MOE_OK
    close("y", y, want["y"], c.H, 0)
    close("n", n, want["n"], c.H, 0)


@pytest.mark.parametrize("how", CASES)
def test_backward(M, monkeypatch, how):
    B, c = M.binding, Case(**how)
    m, want = c.module(M), backward64(c, c.x)
    monkeypatch.setenv("MOE_MXQ_DEBUG_INJECT_WAIT", "1")
    t0 = time.perf_counter()
    m.backward(c.x, c.b, c.gate, c.dy, c.dn)
    assert m.device_status() == B.MOE_ERR_TIMEOUT
    assert time.perf_counter() - t0 < 5.0
    monkeypatch.delenv("MOE_MXQ_DEBUG_INJECT_WAIT")
    got = m.backward(c.x, c.b, c.gate, c.dy, c.dn)
    assert m.device_status() == B.MOE_OK
    for k in want:
        close(k, got[k].reshape(want[k][0].shape), want[k], c.H, c.T)


def test_status_of_calls_through_the_binding(M, monkeypatch):
    """The words are the caller's; without them the NaN alone tell."""
    B, c = M.binding, Case(5, 64)
    y, n, words = torch.empty_like(c.x), torch.empty_like(c.b), torch.full((64,), 9, dtype=torch.uint8, device="cuda")
    monkeypatch.setenv("MOE_MXQ_DEBUG_INJECT_WAIT", "1")
    B.moe_norm_forward(c.x, c.b, None, c.w_post, c.w_pre, y, n)
    assert bool(n[0].isnan().all())
    B.moe_norm_forward(c.x, c.b, None, c.w_post, c.w_pre, y, n, status=words)
    assert B.moe_get_device_status(words) == B.MOE_ERR_TIMEOUT
    monkeypatch.delenv("MOE_MXQ_DEBUG_INJECT_WAIT")
    B.moe_norm_forward(c.x, c.b, None, c.w_post, c.w_pre, y, n, status=words)
    assert not bool(words.any()) and bool(n.isfinite().all())
    words.fill_(9)
    B.moe_norm_forward(c.x[:0], c.b[:0], None, c.w_post, c.w_pre, y[:0], n[:0], status=words)
    assert not bool(words.any())
    assert B.moe_norm_forward(c.x, c.b, None, c.w_post, c.w_pre, y, n, status=words[1:], check=False) == B.MOE_ERR_INVALID_ARG
