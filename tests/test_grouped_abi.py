"""Host-side refusals of the BF16 products grouped by expert (every case returns before the first CUDA call)."""
import ctypes

import pytest
import torch

from tests import helpers as Hp


def _p(v):
    return ctypes.c_void_p(v)


OK = dict(x=0x10000, ldx=64, w=0x20000, offsets=0x30000, P=16, N=128, K=64, E=4, y=0x40000, ldy=128, ws=0x50000, bytes=256)
BAD = [
    (dict(P=-1), "INVALID_ARG"), (dict(N=0), "INVALID_ARG"), (dict(K=-8), "INVALID_ARG"), (dict(E=0), "INVALID_ARG"),
    (dict(N=132), "UNSUPPORTED_SHAPE"), (dict(K=60), "UNSUPPORTED_SHAPE"), (dict(E=1025), "UNSUPPORTED_SHAPE"),
    (dict(P=1 << 31), "UNSUPPORTED_SHAPE"),
    (dict(x=0), "INVALID_ARG"), (dict(w=0), "INVALID_ARG"), (dict(offsets=0), "INVALID_ARG"), (dict(y=0), "INVALID_ARG"),
    (dict(ws=0), "INVALID_ARG"),
    (dict(x=0x10008), "MISALIGNED"), (dict(w=0x20002), "MISALIGNED"), (dict(y=0x40004), "MISALIGNED"),
    (dict(offsets=0x30002), "MISALIGNED"), (dict(ws=0x50080), "MISALIGNED"),
    (dict(bytes=255), "WORKSPACE_TOO_SMALL"),
    (dict(ldx=56), "INVALID_ARG"), (dict(ldx=68), "UNSUPPORTED_SHAPE"),
    (dict(ldy=120), "INVALID_ARG"), (dict(ldy=132), "UNSUPPORTED_SHAPE"),
]


@pytest.mark.parametrize("change,want", BAD)
def test_rows_refusals(change, want):
    B = Hp.lib()
    a = {**OK, **change}
    code = getattr(B, "MOE_ERR_" + want)
    got = B.lib.moe_grouped_forward(_p(a["x"]), a["ldx"], _p(a["w"]), _p(a["offsets"]), a["P"], a["N"], a["K"], a["E"],
                                    _p(a["y"]), a["ldy"], _p(a["ws"]), a["bytes"], None)
    assert got == code
    got = B.lib.moe_grouped_dgrad(_p(a["y"]), a["ldy"], _p(a["w"]), _p(a["offsets"]), a["P"], a["N"], a["K"], a["E"],
                                  _p(a["x"]), a["ldx"], _p(a["ws"]), a["bytes"], None)
    assert got == code


@pytest.mark.parametrize("change,want", BAD + [(dict(dtype=2), "INVALID_ARG"), (dict(acc=2), "INVALID_ARG"),
                                               (dict(acc=1, dtype=0), "INVALID_ARG")])
def test_weights_refusals(change, want):
    B = Hp.lib()
    a = {**OK, "dtype": 1, "acc": 0, **change}
    got = B.lib.moe_grouped_wgrad(_p(a["y"]), a["ldy"], _p(a["x"]), a["ldx"], _p(a["offsets"]), a["P"], a["N"], a["K"],
                                  a["E"], _p(a["w"]), a["dtype"], a["acc"], _p(a["ws"]), a["bytes"], None)
    assert got == getattr(B, "MOE_ERR_" + want)


def test_workspace_size():
    B = Hp.lib()
    assert B.moe_grouped_workspace_size(16, 128, 64, 4) >= 256
    for bad in ((-1, 8, 8, 1), (1, 0, 8, 1), (1, 8, -8, 1), (1, 8, 8, 0)):
        assert B.moe_grouped_workspace_size(*bad) == 0


def test_binding_refuses_tensors_of_other_types_and_strides():
    """Type, shape and stride are looked at before anything is called (so CPU tensors do)."""
    B = Hp.lib()
    bf = torch.bfloat16
    x, w, y = torch.zeros(6, 64, dtype=bf), torch.zeros(2, 128, 64, dtype=bf), torch.zeros(6, 128, dtype=bf)
    off, ws = torch.zeros(3, dtype=torch.int32), torch.zeros(256, dtype=torch.uint8)
    bad_x = [x.float(), x.half(), torch.zeros(6, 72, dtype=bf), torch.zeros(64, 6, dtype=bf).T]
    for t in bad_x:
        assert B.moe_grouped_forward(t, w, off, y, ws, stream=0, check=False) == B.MOE_ERR_INVALID_ARG
        assert B.moe_grouped_dgrad(y, w, off, t, ws, stream=0, check=False) == B.MOE_ERR_INVALID_ARG
        assert B.moe_grouped_wgrad(y, t, off, w, ws, stream=0, check=False) == B.MOE_ERR_INVALID_ARG
    for t in (w.float(), w.transpose(1, 2).contiguous().transpose(1, 2)):
        assert B.moe_grouped_forward(x, t, off, y, ws, stream=0, check=False) == B.MOE_ERR_INVALID_ARG
    for t in (off.long(), off[:2], torch.zeros(6, dtype=torch.int32)[::2]):
        assert B.moe_grouped_forward(x, w, t, y, ws, stream=0, check=False) == B.MOE_ERR_INVALID_ARG
    with pytest.raises(B.MoeError):
        B.moe_grouped_wgrad(y, x, off, w.half(), ws, stream=0)
