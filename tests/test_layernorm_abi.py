"""Host-side refusals of layer norm's calls (every case returns before the first CUDA call)."""
import ctypes

import pytest
import torch

from tests import helpers as Hp

SIZES = dict(struct_size=None, x_dtype=0, w_dtype=1, eps=1e-5, T=16, H=64, w=0x50000)
FORWARD = dict(SIZES, x=0x10000, ldx=64, b=0x20000, ldb=64, bias=0x60000, s=0x30000, lds=64, n=0x40000, ldn=64)
BACKWARD = dict(SIZES, s=0x10000, lds=64, dn=0x20000, ld_dn=64, ds=0x30000, ld_ds=64, dx=0x40000, ld_dx=64, dw=0x60000, dbias=0x70000,
                workspace=0x80000, workspace_bytes=1 << 24)
BAD = [
    (dict(struct_size=8), "INVALID_ARG"), (dict(x_dtype=2), "INVALID_ARG"), (dict(w_dtype=-1), "INVALID_ARG"),
    (dict(eps=-1.0), "INVALID_ARG"), (dict(eps=float("nan")), "INVALID_ARG"), (dict(eps=float("inf")), "INVALID_ARG"),
    (dict(T=-1), "INVALID_ARG"), (dict(H=0), "INVALID_ARG"), (dict(H=60), "UNSUPPORTED_SHAPE"), (dict(H=16392), "UNSUPPORTED_SHAPE"),
    (dict(s=0x10008), "MISALIGNED"), (dict(w=0x50004), "MISALIGNED"), (dict(lds=56), "INVALID_ARG"), (dict(lds=68), "UNSUPPORTED_SHAPE"),
]


def call(B, name, kind, base, change):
    v = {**base, **change}
    v["struct_size"] = v["struct_size"] or ctypes.sizeof(kind)
    return getattr(B.lib, name)(ctypes.byref(kind(**v)), None)


@pytest.mark.parametrize("change,want", BAD + [
    (dict(x=0), "INVALID_ARG"), (dict(n=0), "INVALID_ARG"), (dict(b=0), "INVALID_ARG"), (dict(x=0x10008), "MISALIGNED"),
    (dict(b=0x20002), "MISALIGNED"), (dict(n=0x40008), "MISALIGNED"), (dict(bias=0x60008), "MISALIGNED"), (dict(ldx=56), "INVALID_ARG"),
    (dict(ldb=68), "UNSUPPORTED_SHAPE"), (dict(ldn=63), "INVALID_ARG")])
def test_forward_refusals(change, want):
    B = Hp.lib()
    assert call(B, "moe_layernorm_forward", B.MoeLayernormArgs, FORWARD, change) == getattr(B, "MOE_ERR_" + want)


@pytest.mark.parametrize("change,want", BAD + [
    (dict(s=0), "INVALID_ARG"), (dict(dn=0), "INVALID_ARG"), (dict(w=0), "INVALID_ARG"), (dict(workspace=0), "INVALID_ARG"),
    (dict(workspace=0x80080), "MISALIGNED"), (dict(workspace_bytes=511), "WORKSPACE_TOO_SMALL"), (dict(dn=0x20008), "MISALIGNED"),
    (dict(ds=0x30008), "MISALIGNED"), (dict(dx=0x40008), "MISALIGNED"), (dict(dw=0x60004), "MISALIGNED"), (dict(dbias=0x70008), "MISALIGNED"),
    (dict(ld_dn=56), "INVALID_ARG"), (dict(ld_ds=68), "UNSUPPORTED_SHAPE"), (dict(ld_dx=60), "INVALID_ARG")])
def test_backward_refusals(change, want):
    B = Hp.lib()
    assert call(B, "moe_layernorm_backward", B.MoeLayernormGrads, BACKWARD, change) == getattr(B, "MOE_ERR_" + want)


def test_nothing_to_do_and_no_arguments():
    B = Hp.lib()
    assert call(B, "moe_layernorm_forward", B.MoeLayernormArgs, FORWARD, dict(T=0)) == B.MOE_OK
    assert call(B, "moe_layernorm_backward", B.MoeLayernormGrads, BACKWARD, dict(dx=0, dw=0, dbias=0)) == B.MOE_OK
    assert B.lib.moe_layernorm_forward(None, None) == B.lib.moe_layernorm_backward(None, None) == B.MOE_ERR_INVALID_ARG


def test_workspace_size():
    B = Hp.lib()
    assert B.moe_layernorm_workspace_size(16, 64) >= 16 * 2 * 64 * 4 and B.moe_layernorm_workspace_size(0, 64) >= 512
    for bad in ((-1, 64), (1, 0), (1, 16392)):
        assert B.moe_layernorm_workspace_size(*bad) == 0


def test_binding_refuses_tensors_of_other_types_shapes_and_places():
    B = Hp.lib()
    bf = torch.bfloat16
    x, w, ws = torch.zeros(6, 64, dtype=bf), torch.zeros(64), torch.zeros(1 << 16, dtype=torch.uint8)
    good = dict(x=x, b=x, w=w, bias=w, s=x, n=x)
    for change in ({}, {"x": x.half()}, {"x": x[0]}, {"x": x.float()}, {"b": x.float()}, {"b": x[:5]}, {"w": w[:8]}, {"w": w.half()},
                   {"bias": w.to(bf)}, {"w": torch.zeros(128)[::2]}, {"s": x.float()}, {"n": x.float()}, {"n": torch.zeros(64, 6, dtype=bf).T}):
        assert B.moe_layernorm_forward(**{**good, **change}, stream=0, check=False) == B.MOE_ERR_INVALID_ARG
    good = dict(s=x, w=w, dn=x, ds=x, workspace=ws, dx=x, dw=w, dbias=w)
    for change in ({}, {"s": x.half()}, {"dn": x.float()}, {"ds": x.float()}, {"dx": x.float()}, {"dw": w.to(bf)}, {"dbias": w[:8]},
                   {"w": w[:8]}, {"s": x.float()}):
        assert B.moe_layernorm_backward(**{**good, **change}, stream=0, check=False) == B.MOE_ERR_INVALID_ARG
    with pytest.raises(B.MoeError):
        B.moe_layernorm_forward(**{**FORWARD_TENSORS, "x": x}, stream=0)


FORWARD_TENSORS = dict(b=None, w=None, bias=None, s=None, n=torch.zeros(6, 64, dtype=torch.bfloat16))
