"""The memory that BlockNorm's backward calls write: one's own for each call, as large as it needs, and given back."""
import weakref

import pytest
import torch

from tests import helpers as Hp


@pytest.fixture
def calls(monkeypatch):
    """(BlockNorm, the workspaces given to the library so far); the library's calls are replaced, so no GPU is needed."""
    B = Hp.lib()
    from moe_expert_layer_counting_gb300 import BlockNorm
    given = []

    def backward(y, b, gate, w_post, w_pre, dy, dn, workspace, *outputs_and_how):
        assert workspace.nbytes >= B.moe_norm_workspace_size(*y.shape)
        given.append(workspace)

    monkeypatch.setattr(B, "moe_norm_backward", backward)
    monkeypatch.setattr(B, "_stream", lambda stream: 0)
    return BlockNorm, given


def backward(norm, T, H, gate=None):
    y, b = torch.zeros(T, H, dtype=torch.bfloat16), torch.zeros(T, H, dtype=torch.bfloat16)
    return norm.backward(y, b, gate, y, None)


def test_no_two_calls_share_memory(calls):
    """Two captured graphs, or a graph and a later call, may run at the same time."""
    BlockNorm, given = calls
    norm = BlockNorm()
    for T, H in ((300, 64), (300, 64), (7, 64), (300, 64)):
        backward(norm, T, H)
    spans = sorted((w.data_ptr(), w.data_ptr() + w.nbytes) for w in given)
    assert all(a[1] <= b[0] for a, b in zip(spans, spans[1:]))


def test_rows_of_another_width(calls):
    """Without weights one object serves rows of any length: 64 x 512, then 64 x 1024."""
    BlockNorm, given = calls
    norm = BlockNorm(residual_scale=0.5)
    for H in (512, 1024, 512):
        backward(norm, 64, H)


def test_longer_and_longer_calls_hold_one_workspace(calls):
    BlockNorm, given = calls
    norm, refs = BlockNorm(), []
    for T in range(1, 100):
        backward(norm, T, 64)
        refs.append(weakref.ref(given.pop()))
    assert sum(r() is not None for r in refs) == 1


@pytest.mark.gpu
def test_two_graphs_of_one_object_at_the_same_time():
    """Both captured on torch's capture stream, then replayed side by side: the bits of calls that ran alone."""
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    Hp.lib()
    from moe_expert_layer_counting_gb300 import BlockNorm
    from tests.test_gpu_norm import Case
    cases = [Case(60, 8192, gate="channel", seed=s) for s in (1, 2)]
    norm = BlockNorm(torch.ones(8192, device="cuda"), torch.ones(8192, device="cuda"))

    def call(c):
        return norm.backward(c.x, c.b, c.gate, c.dy, c.dn)

    alone, graphs, outs = [call(c) for c in cases], [], []
    torch.cuda.synchronize()
    for c in cases:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(call(c))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(100):
        for o in outs:
            for t in o.values():
                t.zero_()
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for want, got in zip(alone, outs):
            assert all(torch.equal(want[k], got[k]) for k in want)


@pytest.mark.gpu
def test_widths_and_lengths_on_one_object():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    Hp.lib()
    from moe_expert_layer_counting_gb300 import BlockNorm
    from tests.test_gpu_norm import Case, backward64, close
    norm = BlockNorm(residual_scale=0.75)
    held = []
    for T, H in ((64, 512), (64, 1024), (400, 264), (64, 9000), (1, 8)):
        c = Case(T, H, gate="channel", post=False, pre=False)
        got, want = norm.backward(c.x, c.b, c.gate, c.dy, None), backward64(c, c.x)
        for k in want:
            close(k, got[k], want[k], H, T)
    assert norm.device_status() == 0
    x = torch.zeros(700, 64, dtype=torch.bfloat16, device="cuda")
    for T in range(1, 700):
        norm.backward(x[:T], x[:T], None, x[:T], None)
        held.append(torch.cuda.memory_allocated())
    assert max(held) - min(held) < 1 << 20


def test_refused_status_words():
    """Forward's status words: 4-byte aligned (looked at before anything is enqueued)."""
    from tests.test_norm_abi import args_of
    import ctypes
    B = Hp.lib()
    for T in (0, 4):
        assert B.lib.moe_norm_forward(ctypes.byref(args_of(B, T=T, status=0x8002)), None) == B.MOE_ERR_MISALIGNED


def test_calls_with_nothing_to_compute():
    """Without a layer's answer the stream is x itself: no weight, no n; no dn, and dx is dy.  No GPU is needed."""
    Hp.lib()
    from moe_expert_layer_counting_gb300 import BlockNorm
    x, dy = torch.zeros(3, 64, dtype=torch.bfloat16), torch.ones(3, 64, dtype=torch.bfloat16)
    assert BlockNorm().forward(x) == (x, None)
    for w in (None, torch.ones(64)):
        got = BlockNorm(w_pre=w).backward(x, None, None, dy, None)
        assert got["dx"] is dy and got["db"] is got["dgate"] is got["dw_post"] is got["dw_pre"] is None
        got = BlockNorm(w_pre=w).backward(x, None, None, None, None)
        assert got["dx"].shape == x.shape and got["dx"].dtype is x.dtype and not bool(got["dx"].any())
