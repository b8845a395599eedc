"""Host-side refusals and struct layout of the norms around the layer (nothing here reaches a CUDA call)."""
import ctypes
import os
import shutil
import subprocess

import pytest
import torch

from tests import helpers as Hp

OK = dict(x_dtype=0, w_dtype=1, gate_dtype=1, gate_kind=3, gate_sigmoid=0, residual_scale=1.0, weight_offset=0.0, eps=1e-6, T=4,
          H=64, x=0x1000, ldx=64, b=0x2000, ldb=64, gate=0x3000, ld_gate=64, w_post=0x4000, w_pre=0x5000, y=0x6000, ldy=64,
          n=0x7000, ldn=64)
GRADS = dict(dy=0x10000, ld_dy=64, dn=0x11000, ld_dn=64, dx=0x12000, ld_dx=64, db=0x13000, ld_db=64, dgate=0x14000, ld_dgate=64,
             dw_post=0x15000, dw_pre=0x16000, workspace=0x20000, workspace_bytes=1 << 20)
BAD = [
    (dict(T=-1), "INVALID_ARG"), (dict(H=0), "INVALID_ARG"), (dict(H=60), "UNSUPPORTED_SHAPE"),
    (dict(H=16392, ldx=16392), "UNSUPPORTED_SHAPE"), (dict(T=1 << 31), "UNSUPPORTED_SHAPE"),
    (dict(x_dtype=2), "INVALID_ARG"), (dict(w_dtype=-1), "INVALID_ARG"), (dict(gate_dtype=7), "INVALID_ARG"),
    (dict(gate_kind=4), "INVALID_ARG"), (dict(gate_kind=0), "INVALID_ARG"), (dict(gate=None), "INVALID_ARG"),
    (dict(gate_sigmoid=2), "INVALID_ARG"), (dict(eps=-1.0), "INVALID_ARG"), (dict(eps=float("nan")), "INVALID_ARG"),
    (dict(x=None), "INVALID_ARG"), (dict(b=None), "INVALID_ARG"),
    (dict(ldx=56), "INVALID_ARG"), (dict(ldb=68), "UNSUPPORTED_SHAPE"), (dict(ld_gate=8), "INVALID_ARG"),
    (dict(x=0x1008), "MISALIGNED"), (dict(b=0x2002), "MISALIGNED"), (dict(gate=0x3004), "MISALIGNED"),
    (dict(w_post=0x4004), "MISALIGNED"), (dict(w_pre=0x5008), "MISALIGNED"),
    (dict(gate_kind=1, gate=0x3002), "MISALIGNED"),
]


def args_of(B, **change):
    return B.MoeNormArgs(ctypes.sizeof(B.MoeNormArgs), **{**OK, **change})


def grads_of(B, **change):
    return B.MoeNormGrads(ctypes.sizeof(B.MoeNormGrads), **{**GRADS, **change})


@pytest.mark.parametrize("change,want", BAD)
def test_refusals_of_both(change, want):
    B = Hp.lib()
    code = getattr(B, "MOE_ERR_" + want)
    assert B.lib.moe_norm_forward(ctypes.byref(args_of(B, **change)), None) == code
    assert B.lib.moe_norm_backward(ctypes.byref(args_of(B, **change)), ctypes.byref(grads_of(B)), None) == code


@pytest.mark.parametrize("change,want", [
    (dict(n=None), "INVALID_ARG"), (dict(w_pre=None), "INVALID_ARG"), (dict(w_pre=None, n=None, y=None), "INVALID_ARG"),
    (dict(b=None, gate=None, gate_kind=0, w_post=None), "INVALID_ARG"),            # y without b
    (dict(y=0x6008), "MISALIGNED"), (dict(n=0x7004), "MISALIGNED"), (dict(ldy=40), "INVALID_ARG"),
    (dict(ldn=66), "UNSUPPORTED_SHAPE")])
def test_forward_refusals(change, want):
    B = Hp.lib()
    assert B.lib.moe_norm_forward(ctypes.byref(args_of(B, **change)), None) == getattr(B, "MOE_ERR_" + want)


@pytest.mark.parametrize("change,want,of_args", [
    (dict(dn=None), "INVALID_ARG", {}), (dict(), "INVALID_ARG", dict(w_pre=None)),
    (dict(dw_post=0x15000), "INVALID_ARG", dict(w_post=None)),
    (dict(dgate=0x14000), "INVALID_ARG", dict(gate=None, gate_kind=0)),
    (dict(workspace=None), "INVALID_ARG", {}), (dict(workspace=0x20010), "MISALIGNED", {}),
    (dict(workspace_bytes=100), "WORKSPACE_TOO_SMALL", {}),
    (dict(dy=0x10008), "MISALIGNED", {}), (dict(dx=0x12004), "MISALIGNED", {}), (dict(ld_db=70), "UNSUPPORTED_SHAPE", {}),
    (dict(ld_dn=0), "INVALID_ARG", {}), (dict(ld_dgate=32), "INVALID_ARG", {}), (dict(dw_pre=0x16004), "MISALIGNED", {})])
def test_backward_refusals(change, want, of_args):
    B = Hp.lib()
    got = B.lib.moe_norm_backward(ctypes.byref(args_of(B, **of_args)), ctypes.byref(grads_of(B, **change)), None)
    assert got == getattr(B, "MOE_ERR_" + want)


def test_struct_size_and_no_rows():
    B = Hp.lib()
    a, g = args_of(B), grads_of(B)
    a.struct_size -= 8
    assert B.lib.moe_norm_forward(ctypes.byref(a), None) == B.MOE_ERR_INVALID_ARG
    a, g.struct_size = args_of(B), 0
    assert B.lib.moe_norm_backward(ctypes.byref(a), ctypes.byref(g), None) == B.MOE_ERR_INVALID_ARG
    assert B.lib.moe_norm_forward(None, None) == B.MOE_ERR_INVALID_ARG
    assert B.lib.moe_norm_forward(ctypes.byref(args_of(B, T=0)), None) == B.MOE_OK
    assert B.moe_norm_workspace_size(-1, 64) == 0 and B.moe_norm_workspace_size(4, 0) == 0
    assert B.moe_norm_workspace_size(4, 64) >= 4 * 2 * 64 * 4


def test_struct_layout_matches_c(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if not cc:
        pytest.skip("no C compiler")
    B = Hp.lib()
    names = [("moe_norm_args", B.MoeNormArgs), ("moe_norm_grads", B.MoeNormGrads)]
    lines = "".join(f'printf("%zu\\n", sizeof({n}));' + "".join(f'printf("%zu\\n", offsetof({n}, {f[0]}));' for f in s._fields_)
                    for n, s in names)
    (tmp_path / "l.c").write_text('#include <stdio.h>\n#include <stddef.h>\n#include "moe_norm.h"\nint main(void){%s return 0;}'
                                  % lines)
    subprocess.run([cc, "-I", os.path.join(Hp.ROOT, "include"), str(tmp_path / "l.c"), "-o", str(tmp_path / "l")], check=True)
    got = [int(v) for v in subprocess.run([str(tmp_path / "l")], capture_output=True, text=True, check=True).stdout.split()]
    assert got == [v for _, s in names for v in (ctypes.sizeof(s), *(getattr(s, f[0]).offset for f in s._fields_))]


def test_binding_refuses_tensors_of_other_types_and_shapes():
    B = Hp.lib()
    bf = torch.bfloat16
    x, b, w = torch.zeros(3, 64, dtype=bf), torch.zeros(3, 64, dtype=bf), torch.ones(64)

    def call(x=x, b=b, gate=None, w_post=w, w_pre=w, y=x, n=b):
        return B.moe_norm_forward(x, b, gate, w_post, w_pre, y, n, stream=0, check=False)

    bad = [dict(x=x.half()), dict(b=b.float()), dict(y=x.float()), dict(n=torch.zeros(3, 72, dtype=bf)),
           dict(x=torch.zeros(64, 3, dtype=bf).T), dict(w_pre=w.double()), dict(w_pre=w.to(bf)), dict(w_post=torch.ones(32)),
           dict(gate=torch.zeros(3)), dict(gate=torch.zeros(2, 1)), dict(gate=torch.zeros(3, 64, dtype=torch.half)),
           dict(gate=torch.zeros(64, 3).T)]
    for change in bad:
        assert call(**change) == B.MOE_ERR_INVALID_ARG, change
    with pytest.raises(B.MoeError):
        B.moe_norm_forward(x.half(), b, None, w, w, x, b, stream=0)
