"""Host-side refusals and struct layout of the AdamW step (nothing here reaches a CUDA call)."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

from tests import helpers as Hp

ARGS = dict(p_dtype=1, g_dtype=0, state_bits=8, grad_scale=0x90000, lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1,
            step=1)
TENSOR = dict(n=100, p=0x10000, g=0x20000, m=0x30000, v=0x40000, m_scale=0x50001, v_scale=0x60003, copy=0x70000)


def call(B, tensor=None, n_tensors=1, **change):
    table = np.zeros(max(1, n_tensors), B.ADAMW_TENSOR)
    for k, v in {**TENSOR, **(tensor or {})}.items():
        table[k] = v
    a = B.MoeAdamwArgs(ctypes.sizeof(B.MoeAdamwArgs), n_tensors, table.ctypes.data, **{**ARGS, **change})
    return B.lib.moe_adamw_step(ctypes.byref(a), None)


@pytest.mark.parametrize("change", [
    dict(p_dtype=2), dict(g_dtype=-1), dict(state_bits=16), dict(step=0), dict(beta1=1.0), dict(beta1=-0.1), dict(beta2=1.0),
    dict(eps=-1e-8), dict(eps=float("inf")), dict(lr=float("nan")), dict(weight_decay=float("inf")), dict(beta2=float("nan")),
    dict(n_tensors=-1)])
def test_refused_arguments(change):
    B = Hp.lib()
    assert call(B, **change) == B.MOE_ERR_INVALID_ARG


@pytest.mark.parametrize("tensor,want,change", [
    (dict(n=-1), "INVALID_ARG", {}), (dict(p=0), "INVALID_ARG", {}), (dict(g=0), "INVALID_ARG", {}),
    (dict(m=0), "INVALID_ARG", {}), (dict(v=0), "INVALID_ARG", {}), (dict(m_scale=0), "INVALID_ARG", {}),
    (dict(v_scale=0), "INVALID_ARG", {}), (dict(), "INVALID_ARG", dict(p_dtype=0)),      # a copy of a BF16 p
    (dict(p=0x10004), "MISALIGNED", {}), (dict(g=0x20008), "MISALIGNED", {}), (dict(m=0x30001), "MISALIGNED", {}),
    (dict(v=0x40008), "MISALIGNED", {}), (dict(copy=0x70002), "MISALIGNED", {}),
    (dict(), "MISALIGNED", dict(grad_scale=0x90002)), (dict(n=1 << 62), "UNSUPPORTED_SHAPE", {})])
def test_refused_tensors(tensor, want, change):
    B = Hp.lib()
    assert call(B, tensor, **change) == getattr(B, "MOE_ERR_" + want)


def test_nothing_to_do():
    B = Hp.lib()
    assert call(B, n_tensors=0) == B.MOE_OK
    assert call(B, dict(n=0, p=0, g=0, m=0, v=0), n_tensors=3) == B.MOE_OK
    a = B.MoeAdamwArgs(8, 0, None, **ARGS)
    assert B.lib.moe_adamw_step(ctypes.byref(a), None) == B.MOE_ERR_INVALID_ARG
    assert B.lib.moe_adamw_step(None, None) == B.MOE_ERR_INVALID_ARG


def test_struct_layout_matches_c(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if not cc:
        pytest.skip("no C compiler")
    B = Hp.lib()
    fields = [f[0] for f in B.MoeAdamwArgs._fields_]
    body = "".join(f'printf("%zu\\n", offsetof(moe_adamw_args, {f}));' for f in fields) + \
        "".join(f'printf("%zu\\n", offsetof(moe_adamw_tensor, {f}));' for f in B.ADAMW_TENSOR.names)
    (tmp_path / "l.c").write_text('#include <stdio.h>\n#include <stddef.h>\n#include "moe_adamw.h"\nint main(void){'
                                  'printf("%%zu %%zu\\n", sizeof(moe_adamw_args), sizeof(moe_adamw_tensor)); %s return 0;}' % body)
    subprocess.run([cc, "-I", os.path.join(Hp.ROOT, "include"), str(tmp_path / "l.c"), "-o", str(tmp_path / "l")], check=True)
    got = [int(v) for v in subprocess.run([str(tmp_path / "l")], capture_output=True, text=True, check=True).stdout.split()]
    assert got == [ctypes.sizeof(B.MoeAdamwArgs), B.ADAMW_TENSOR.itemsize,
                   *(getattr(B.MoeAdamwArgs, f).offset for f in fields),
                   *(B.ADAMW_TENSOR.fields[f][1] for f in B.ADAMW_TENSOR.names)]


def test_the_optimizer_refuses_tensors_that_do_not_fit():
    Hp.lib()
    from moe_expert_layer_counting_gb300 import AdamW, binding as B
    p = [torch.zeros(4, 8), torch.zeros(40)]
    for bad in (dict(state_bits=16), dict(copies=[torch.zeros(32)] * 2), dict(copies=[torch.zeros(32, dtype=torch.bfloat16)] * 2),
                dict(state=([torch.zeros(32), torch.zeros(41)], [torch.zeros(32), torch.zeros(40)])),
                dict(state=([torch.zeros(32), torch.zeros(80)[::2]], [torch.zeros(32), torch.zeros(40)]))):
        with pytest.raises(ValueError):
            AdamW(p, **bad)
    with pytest.raises(ValueError):
        AdamW([torch.zeros(4), torch.zeros(4, dtype=torch.bfloat16)])
    with pytest.raises(ValueError):
        AdamW([torch.zeros(8, 4).T])
    opt = AdamW(p)
    for bad in ([torch.zeros(32)], [torch.zeros(32), torch.zeros(41)], [torch.zeros(32), torch.zeros(40, dtype=torch.half)],
                [torch.zeros(32, dtype=torch.bfloat16), torch.zeros(40)], [torch.zeros(8, 4).T, torch.zeros(40)]):
        with pytest.raises(ValueError):
            opt.step(bad)
    with pytest.raises(B.MoeError):
        B.moe_adamw_step(np.zeros(1, np.int64), 1, 1, 32, 1e-3, 0.9, 0.9, 1e-8, 0.0, 1, stream=0)
