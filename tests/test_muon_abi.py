"""Host-side refusals of the orthogonalisation and of Muon (every case returns before the first CUDA call)."""
import ctypes

import pytest
import torch

from tests import helpers as Hp

NS = dict(steps=5, a=3.4445, b=-4.775, c=2.0315, eps=1e-7)
STACK = dict(struct_size=None, E=2, N=16, K=24, status=0, workspace=0x70000, workspace_bytes=1 << 30)
STEP = dict(STACK, p_dtype=1, g_dtype=0, nesterov=1, p=0x10000, g=0x20000, m=0x30000, copy=0x40000, grad_scale=0x50000, lr=1e-3,
            momentum=0.9, weight_decay=0.1, scale=1.0)
ORTHO = dict(STACK, x_dtype=0, out_dtype=0, x=0x10000, out=0x20000)
NAN, INF = float("nan"), float("inf")
BAD = [
    (dict(struct_size=8), "INVALID_ARG"), (dict(E=-1), "INVALID_ARG"), (dict(N=0), "INVALID_ARG"), (dict(K=-8), "INVALID_ARG"),
    (dict(N=1 << 20), "UNSUPPORTED_SHAPE"), (dict(K=1 << 20), "UNSUPPORTED_SHAPE"), (dict(E=65536), "UNSUPPORTED_SHAPE"),
    (dict(workspace=0), "INVALID_ARG"), (dict(workspace=0x70080), "MISALIGNED"), (dict(workspace_bytes=256), "WORKSPACE_TOO_SMALL"),
    (dict(status=0x60002), "MISALIGNED"),
    (dict(ns=dict(steps=-1)), "INVALID_ARG"), (dict(ns=dict(steps=65)), "INVALID_ARG"), (dict(ns=dict(eps=-1.0)), "INVALID_ARG"),
    (dict(ns=dict(eps=NAN)), "INVALID_ARG"), (dict(ns=dict(eps=INF)), "INVALID_ARG"), (dict(ns=dict(a=NAN)), "INVALID_ARG"),
    (dict(ns=dict(b=65.0)), "INVALID_ARG"), (dict(ns=dict(c=-INF)), "INVALID_ARG"), (dict(ns=dict(c=0.1)), "INVALID_ARG"),
]


def call(B, name, kind, base, change):
    v = {**base, **change}
    v["ns"] = B.MoeNewtonSchulz(**{**NS, **change.get("ns", {})})
    v["struct_size"] = v["struct_size"] or ctypes.sizeof(kind)
    return getattr(B.lib, name)(ctypes.byref(kind(**v)), None)


@pytest.mark.parametrize("change,want", BAD + [
    (dict(p_dtype=2), "INVALID_ARG"), (dict(g_dtype=-1), "INVALID_ARG"), (dict(nesterov=2), "INVALID_ARG"),
    (dict(lr=INF), "INVALID_ARG"), (dict(momentum=1.0), "INVALID_ARG"), (dict(momentum=-0.1), "INVALID_ARG"),
    (dict(momentum=NAN), "INVALID_ARG"), (dict(weight_decay=NAN), "INVALID_ARG"), (dict(scale=INF), "INVALID_ARG"),
    (dict(p=0), "INVALID_ARG"), (dict(g=0), "INVALID_ARG"), (dict(m=0), "INVALID_ARG"),
    (dict(p=0x10002), "MISALIGNED"), (dict(g=0x20001), "MISALIGNED"), (dict(m=0x30002), "MISALIGNED"),
    (dict(copy=0x40001), "MISALIGNED"), (dict(grad_scale=0x50002), "MISALIGNED")])
def test_step_refusals(change, want):
    B = Hp.lib()
    assert call(B, "moe_muon_step", B.MoeMuonArgs, STEP, change) == getattr(B, "MOE_ERR_" + want)


@pytest.mark.parametrize("change,want", BAD + [
    (dict(x_dtype=2), "INVALID_ARG"), (dict(out_dtype=2), "INVALID_ARG"), (dict(x=0), "INVALID_ARG"), (dict(out=0), "INVALID_ARG"),
    (dict(x=0x10001), "MISALIGNED"), (dict(out=0x20002, out_dtype=1), "MISALIGNED")])
def test_orthogonalize_refusals(change, want):
    B = Hp.lib()
    assert call(B, "moe_orthogonalize", B.MoeOrthogonalizeArgs, ORTHO, change) == getattr(B, "MOE_ERR_" + want)


def test_no_matrices_and_no_arguments():
    B = Hp.lib()
    empty = dict(E=0, workspace=0, workspace_bytes=0)
    assert call(B, "moe_muon_step", B.MoeMuonArgs, STEP, empty) == B.MOE_OK
    assert call(B, "moe_orthogonalize", B.MoeOrthogonalizeArgs, ORTHO, empty) == B.MOE_OK
    assert B.lib.moe_muon_step(None, None) == B.lib.moe_orthogonalize(None, None) == B.MOE_ERR_INVALID_ARG


def test_workspace_size():
    B = Hp.lib()
    # two iterates, S and Q in FP16
    assert B.moe_muon_workspace_size(3, 100, 52) >= 256 + 3 * 2 * (2 * 100 * 56 + 2 * 52 * 56)
    for bad in ((-1, 8, 8), (1, 0, 8), (1, 8, -8), (1, 1 << 20, 8), (65536, 8, 8)):
        assert B.moe_muon_workspace_size(*bad) == 0


def test_binding_refuses_tensors_of_other_types_shapes_and_places():
    B = Hp.lib()
    x = torch.zeros(2, 16, 24)
    ws = torch.zeros(1 << 16, dtype=torch.uint8)
    for a, o in ((x, x), (x.half(), x), (x, x.half()), (x, x[:1]), (x.transpose(1, 2), x.transpose(1, 2)), (x[0, 0], x[0, 0])):
        assert B.moe_orthogonalize(a, o, ws, stream=0, check=False) == B.MOE_ERR_INVALID_ARG      # the first: of the CPU
    good = dict(p=x, g=x, m=x, workspace=ws, lr=0.1)
    for change in ({}, {"p": x.double()}, {"g": x[:, :8]}, {"m": x.bfloat16()}, {"copy": x}, {"grad_scale": torch.zeros(2)},
                   {"grad_scale": torch.zeros(1, dtype=torch.float64)}, {"status": torch.zeros(32, dtype=torch.uint8)}):
        assert B.moe_muon_step(**{**good, **change}, stream=0, check=False) == B.MOE_ERR_INVALID_ARG
    with pytest.raises(B.MoeError):
        B.moe_orthogonalize(x, x, ws, stream=0)


@pytest.mark.parametrize("params,more", [
    ([torch.zeros(8)], {}), ([torch.zeros(8, 8).half()], {}), ([torch.zeros(8, 16)[:, :8]], {}), ([torch.zeros(8, 8)], {"adjust": "no"}),
    ([torch.zeros(8, 8)], {"copies": []}), ([torch.zeros(8, 8)], {"copies": [torch.zeros(8, 8)]}),
    ([torch.zeros(8, 8)], {"state": ([torch.zeros(8, 8).bfloat16()],)}), ([torch.zeros(8, 8)], {"state": ([torch.zeros(64)],)}),
    ([torch.zeros(8, 8)], {"state": ([torch.zeros(8, 8)], [torch.zeros(8, 8)])}), ([torch.zeros(8, 8)], {"state": ([None],)})])
def test_object_refusals(params, more):
    Hp.lib()
    from moe_expert_layer_counting_gb300 import Muon
    with pytest.raises(ValueError):
        Muon(params, **more)


def test_step_refuses_other_gradients():
    Hp.lib()
    from moe_expert_layer_counting_gb300 import Muon
    opt = Muon([torch.zeros(8, 16)])
    for grads in ([], [torch.zeros(16, 8)], [torch.zeros(8, 16).half()], [torch.zeros(16, 8).T], [None],
                  [torch.zeros(8, 16, device="meta")]):
        with pytest.raises(ValueError):
            opt.step(grads, stream=0)
    opt.params[0] = torch.zeros(8, 8)          # the momentum is still of the other
    with pytest.raises(ValueError):
        opt.step([torch.zeros(8, 8)], stream=0)
