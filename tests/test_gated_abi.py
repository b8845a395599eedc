"""Host-side refusals of the gated block's calls (every case returns before the first CUDA call)."""
import ctypes

import pytest
import torch

from tests import helpers as Hp

OK = dict(struct_size=None, E=4, activation=0, P=16, H=64, I=128, rows=0x10000, ld_rows=64, w=0x20000, offsets=0x30000,
          row_w=0x30100, a=0x40000, ld_a=256, h=0x50000, ld_h=128, da=0x60000, ld_da=256, drow_w=0x30200, workspace=0x70000,
          workspace_bytes=1 << 20)
BAD = [
    (dict(struct_size=8), "INVALID_ARG"), (dict(P=-1), "INVALID_ARG"), (dict(H=0), "INVALID_ARG"), (dict(I=-8), "INVALID_ARG"),
    (dict(E=0), "INVALID_ARG"), (dict(activation=2), "INVALID_ARG"), (dict(activation=-1), "INVALID_ARG"),
    (dict(H=60), "UNSUPPORTED_SHAPE"), (dict(I=100), "UNSUPPORTED_SHAPE"), (dict(E=1025), "UNSUPPORTED_SHAPE"),
    (dict(P=1 << 31), "UNSUPPORTED_SHAPE"), (dict(I=1 << 30), "UNSUPPORTED_SHAPE"),
    (dict(rows=0), "INVALID_ARG"), (dict(w=0), "INVALID_ARG"), (dict(offsets=0), "INVALID_ARG"),
    (dict(workspace=0), "INVALID_ARG"),
    (dict(rows=0x10008), "MISALIGNED"), (dict(w=0x20002), "MISALIGNED"), (dict(a=0x40004), "MISALIGNED"),
    (dict(h=0x50008), "MISALIGNED"), (dict(offsets=0x30002), "MISALIGNED"), (dict(row_w=0x30102), "MISALIGNED"),
    (dict(workspace=0x70080), "MISALIGNED"), (dict(workspace_bytes=255), "WORKSPACE_TOO_SMALL"),
    (dict(ld_rows=56), "INVALID_ARG"), (dict(ld_rows=68), "UNSUPPORTED_SHAPE"),
    (dict(ld_a=248), "INVALID_ARG"), (dict(ld_a=260), "UNSUPPORTED_SHAPE"),
    (dict(ld_h=120), "INVALID_ARG"), (dict(ld_h=132), "UNSUPPORTED_SHAPE"),
]


def call(B, name, **change):
    v = {**OK, **change}
    a = B.MoeGatedArgs(**{**v, "struct_size": v["struct_size"] or ctypes.sizeof(B.MoeGatedArgs)})
    return getattr(B.lib, name)(ctypes.byref(a), None)


@pytest.mark.parametrize("change,want", BAD + [(dict(h=0), "INVALID_ARG"), (dict(da=0x60000), "INVALID_ARG"),
                                               (dict(drow_w=0x30200), "INVALID_ARG")])
def test_forward_refusals(change, want):
    B = Hp.lib()
    assert call(B, "moe_gated_forward", **{"da": 0, "drow_w": 0, **change}) == getattr(B, "MOE_ERR_" + want)


@pytest.mark.parametrize("change,want", BAD + [(dict(a=0), "INVALID_ARG"), (dict(da=0), "INVALID_ARG"),
                                               (dict(da=0x60008), "MISALIGNED"), (dict(ld_da=248), "INVALID_ARG"),
                                               (dict(ld_da=260), "UNSUPPORTED_SHAPE"), (dict(drow_w=0x30202), "MISALIGNED")])
def test_back_refusals(change, want):
    B = Hp.lib()
    assert call(B, "moe_gated_dgrad", **change) == getattr(B, "MOE_ERR_" + want)


def test_no_arguments():
    B = Hp.lib()
    assert B.lib.moe_gated_forward(None, None) == B.lib.moe_gated_dgrad(None, None) == B.MOE_ERR_INVALID_ARG


def test_workspace_size():
    B = Hp.lib()
    assert B.moe_gated_workspace_size(16, 64, 128, 4) >= 256 + 16 * 4 * 4
    assert B.moe_gated_workspace_size(0, 64, 128, 4) >= 256
    for bad in ((-1, 8, 8, 1), (1, 0, 8, 1), (1, 8, -8, 1), (1, 8, 8, 0)):
        assert B.moe_gated_workspace_size(*bad) == 0


def test_binding_refuses_tensors_of_other_types_shapes_and_places():
    B = Hp.lib()
    bf = torch.bfloat16
    t = {"x": torch.zeros(6, 64, dtype=bf), "w": torch.zeros(2, 256, 64, dtype=bf), "offsets": torch.zeros(3, dtype=torch.int32),
         "h": torch.zeros(6, 128, dtype=bf), "a": torch.zeros(6, 256, dtype=bf), "row_w": torch.zeros(6)}
    ws = torch.zeros(4096, dtype=torch.uint8)
    changes = [{}, {"x": t["x"].float()}, {"x": t["x"][:, :56]}, {"x": torch.zeros(64, 6, dtype=bf).T}, {"w": t["w"].float()},
               {"w": t["w"][0]}, {"w": t["w"][:, :255]}, {"w": t["w"].transpose(1, 2)}, {"offsets": t["offsets"].long()},
               {"offsets": t["offsets"][:2]}, {"h": t["h"][:5]}, {"h": t["h"].half()}, {"a": t["a"][:, :128]},
               {"row_w": t["row_w"].double()}, {"row_w": t["row_w"][:, None]}, {"row_w": torch.zeros(12)[::2]}]
    for change in changes:                # the first one: tensors of the CPU
        v = {**t, **change}
        assert B.moe_gated_forward(v["x"], v["w"], v["offsets"], v["h"], ws, a=v["a"], row_w=v["row_w"], stream=0,
                                   check=False) == B.MOE_ERR_INVALID_ARG
        if "w" not in change:
            down = torch.zeros(2, 64, 128, dtype=bf)
            assert B.moe_gated_dgrad(v["x"], down, v["offsets"], v["a"], torch.zeros(6, 256, dtype=bf), ws, h=v["h"],
                                     row_w=v["row_w"], stream=0, check=False) == B.MOE_ERR_INVALID_ARG
    with pytest.raises(B.MoeError):
        B.moe_gated_forward(t["x"], t["w"], t["offsets"], t["h"], ws, stream=0)


@pytest.mark.parametrize("l1,l2,more", [
    (torch.zeros(256, 64, dtype=torch.bfloat16), torch.zeros(64, 64, dtype=torch.bfloat16), {}),
    (torch.zeros(256, 64), torch.zeros(64, 128), {}),
    (torch.zeros(255, 64, dtype=torch.bfloat16), torch.zeros(64, 127, dtype=torch.bfloat16), {}),
    (torch.zeros(256, 64, dtype=torch.bfloat16), torch.zeros(128, 64, dtype=torch.bfloat16).T, {}),
    (torch.zeros(256, 64, dtype=torch.bfloat16), torch.zeros(64, 128, dtype=torch.bfloat16), {"activation": 3})])
def test_block_refusals(l1, l2, more):
    Hp.lib()
    from moe_expert_layer_counting_gb300 import GatedFeedForward
    with pytest.raises(ValueError):
        GatedFeedForward(l1, l2, **more)


def test_block_refuses_other_rows():
    Hp.lib()
    from moe_expert_layer_counting_gb300 import GatedFeedForward
    block = GatedFeedForward(torch.zeros(256, 64, dtype=torch.bfloat16), torch.zeros(64, 128, dtype=torch.bfloat16))
    for n in (torch.zeros(5, 64), torch.zeros(64, dtype=torch.bfloat16), torch.zeros(5, 72, dtype=torch.bfloat16),
              torch.zeros(5, 64, dtype=torch.bfloat16, device="meta")):
        with pytest.raises(ValueError):
            block.forward(n)
    s = {"n": torch.zeros(5, 64, dtype=torch.bfloat16), "a": None, "h": None, "offsets": None}
    for db in (torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(5, 64)):
        with pytest.raises(ValueError):
            block.backward(db, s, torch.zeros(256, 64), torch.zeros(64, 128))
    with pytest.raises(ValueError):
        block.backward(s["n"], s, torch.zeros(128, 64), torch.zeros(64, 128))
