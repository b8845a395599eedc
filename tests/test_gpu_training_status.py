"""What the training objects report of a device-side wait that ran out in one of a step's calls, when the calls after it were
fine: the first code is the step's.

Only the call under test has its wait injected (the host reads the variable as it enqueues), so that no other workspace holds a
code."""
import os

import pytest
import torch

from tests import helpers as Hp

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def M():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    Hp.lib()
    import moe_expert_layer_counting_gb300 as package
    return package


def randn(*shape, seed=0, scale=1.0, dtype=BF16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def inject(monkeypatch, B, name):
    """Every call of this entry point enqueues a kernel whose first wait runs out."""
    call = getattr(B, name)

    def injected(*args, **kwargs):
        os.environ["MOE_MXQ_DEBUG_INJECT_WAIT"] = "1"
        try:
            return call(*args, **kwargs)
        finally:
            del os.environ["MOE_MXQ_DEBUG_INJECT_WAIT"]

    monkeypatch.setattr(B, name, injected)


def experts_step(M, T=60, E=2, H=128, I=64, k=2):
    layer = M.TrainableExperts(randn(E, 2 * I, H, scale=0.1), randn(E, H, I, scale=0.1), fused=True)
    idx = torch.arange(T * k, dtype=torch.int32, device="cuda").view(T, k) % E
    w = torch.full((T, k), 0.5, device="cuda")
    dl1, dl2 = torch.zeros(E, 2 * I, H, device="cuda"), torch.zeros(E, H, I, device="cuda")

    def forward():
        return layer.forward(randn(T, H, seed=1), idx, w)[1]

    return layer, forward, lambda kept: layer.backward(randn(T, H, seed=2), kept, dl1, dl2)


@pytest.mark.parametrize("name", ["moe_gated_forward", "moe_gated_dgrad"])
def test_fused_experts_report_either_gated_call(M, monkeypatch, name):
    from moe_expert_layer_counting_gb300 import binding as B
    layer, forward, backward = experts_step(M)
    with monkeypatch.context() as m:
        inject(m, B, name)
        backward(forward())
    assert layer.status() == B.MOE_ERR_TIMEOUT
    kept = forward()
    assert layer.status() == (B.MOE_OK if name == "moe_gated_forward" else B.MOE_ERR_TIMEOUT)
    backward(kept)
    assert layer.status() == B.MOE_OK


@pytest.mark.parametrize("name", ["moe_gated_forward", "moe_gated_dgrad"])
def test_a_gated_block_reports_either_gated_call(M, monkeypatch, name):
    from moe_expert_layer_counting_gb300 import binding as B
    T, H, I = 60, 128, 64
    block = M.GatedFeedForward(randn(2 * I, H, scale=0.1), randn(H, I, scale=0.1))
    dl1, dl2 = torch.zeros(2 * I, H, device="cuda"), torch.zeros(H, I, device="cuda")

    def step():
        kept = block.forward(randn(T, H, seed=1))[1]
        block.backward(randn(T, H, seed=2), kept, dl1, dl2)

    with monkeypatch.context() as m:
        inject(m, B, name)
        step()
    assert block.status() == B.MOE_ERR_TIMEOUT
    step()
    assert block.status() == B.MOE_OK


@pytest.mark.parametrize("shape", [(2, 300, 136), (2, 72, 40)])
def test_muon_reports_replayed_steps(M, monkeypatch, shape):
    """A captured step's code is its last replay's, whatever stream the replay ran on, and none before the first replay."""
    from moe_expert_layer_counting_gb300 import binding as B
    p, g = randn(*shape, seed=9, scale=0.02, dtype=torch.float32), randn(*shape, seed=1, scale=1e-3)
    opt = M.Muon([p.clone(), p], lr=0.01)
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for graph in graphs:
        with monkeypatch.context() as m:
            if graph is graphs[0]:
                inject(m, B, "moe_muon_step")
            with torch.cuda.graph(graph):
                opt.step([g, g])
        assert opt.device_status() == B.MOE_OK
    graphs[0].replay()
    assert opt.device_status() == B.MOE_ERR_TIMEOUT
    opt.step([g, g])                                        # an eager step's words are its own
    assert opt.device_status() == B.MOE_ERR_TIMEOUT
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graphs[1].replay()
    torch.cuda.synchronize()
    assert opt.device_status() == opt.device_status(side) == B.MOE_OK


def test_muon_with_more_parameters_is_captured_after_a_step(M):
    """The words of captured steps are made outside of a capture, one for each parameter; graphs of before keep theirs."""
    p, g = randn(2, 72, 40, scale=0.02, dtype=torch.float32), randn(2, 72, 40, seed=1, scale=1e-3)
    opt, graph = M.Muon([p], lr=0.01), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        opt.step([g])
    opt.params.append(p.clone())
    opt.state["m"].append(torch.zeros_like(p))
    before = [t.clone() for t in (*opt.params, *opt.state["m"])]
    with pytest.raises(RuntimeError):
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            opt.step([g, g])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(before, (*opt.params, *opt.state["m"])))
    opt.step([g, g])
    graph.replay()
    with torch.cuda.graph(torch.cuda.CUDAGraph()):
        opt.step([g, g])
    assert opt.device_status() == 0
