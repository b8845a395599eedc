"""Lists of parameters of which one cannot be updated: Muon refuses all of them, so that a refused step has moved none (without a
GPU)."""
import pytest
import torch

from tests import helpers as Hp

BAD = [torch.zeros(8, 16, device="meta"),           # on another device than the first
       torch.zeros(65536, 1, 2),                    # more matrices than a call takes
       torch.zeros(1, 1).expand(1, 1 << 20).contiguous()]      # more columns


@pytest.fixture
def Muon(monkeypatch):
    B = Hp.lib()
    from moe_expert_layer_counting_gb300 import Muon

    def called(*_, **__):
        raise AssertionError("the library was called")

    monkeypatch.setattr(B, "moe_muon_step", called)
    return Muon


@pytest.mark.parametrize("bad", BAD)
def test_at_the_start(Muon, bad):
    with pytest.raises(ValueError):
        Muon([torch.zeros(8, 16), bad])


@pytest.mark.parametrize("bad", BAD)
def test_at_a_step(Muon, bad, monkeypatch):
    opt = Muon([torch.zeros(8, 16), torch.zeros(8, 16)])
    opt.params[1], opt.state["m"][1] = bad, torch.zeros_like(bad, dtype=torch.float32)
    with pytest.raises(ValueError):
        opt.step([torch.zeros(8, 16), torch.zeros_like(bad)], stream=0)

