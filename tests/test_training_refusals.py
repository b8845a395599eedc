"""What TrainableExperts refuses, before the library or an index operation sees it (so without a GPU)."""
import pytest
import torch

from tests import helpers as Hp

T, E, H, I, k = 5, 4, 64, 32, 2
BF16 = torch.bfloat16


@pytest.fixture
def layer(monkeypatch):
    B = Hp.lib()
    from moe_expert_layer_counting_gb300.training import TrainableExperts

    def called(*_, **__):
        raise AssertionError("the library was called")

    for name in ("moe_permute", "moe_grouped_forward", "moe_grouped_dgrad", "moe_grouped_wgrad", "moe_combine"):
        monkeypatch.setattr(B, name, called)
    return TrainableExperts(torch.zeros(E, 2 * I, H, dtype=BF16), torch.zeros(E, H, I, dtype=BF16))


@pytest.mark.parametrize("change", [
    dict(idx=torch.zeros(T, k, dtype=torch.int64)), dict(idx=torch.zeros(T * k, dtype=torch.int32)),
    dict(idx=torch.zeros(T, k)), dict(idx=torch.zeros(T, k, dtype=torch.int32, device="meta")),
    dict(n=torch.zeros(T - 1, H, dtype=BF16)), dict(n=torch.zeros(T + 1, H, dtype=BF16)), dict(n=torch.zeros(T, H)),
    dict(n=torch.zeros(T, H + 8, dtype=BF16)), dict(n=torch.zeros(T, H, dtype=BF16, device="meta")),
    dict(w=torch.zeros(T, k - 1)), dict(w=torch.zeros(T - 1, k)), dict(w=torch.zeros(k, T))])
def test_forward(layer, change):
    a = {"n": torch.zeros(T, H, dtype=BF16), "idx": torch.zeros(T, k, dtype=torch.int32), "w": torch.zeros(T, k), **change}
    with pytest.raises(ValueError):
        layer.forward(a["n"], a["idx"], a["w"])


@pytest.mark.parametrize("db", [torch.zeros(T - 1, H, dtype=BF16), torch.zeros(T, H), torch.zeros(T, H - 8, dtype=BF16),
                                torch.zeros(T, H, dtype=BF16, device="meta")])
def test_backward(layer, db):
    s = {"row": torch.zeros(T, k, dtype=torch.int32), "token": torch.zeros(T * k, dtype=torch.int64),
         "h": torch.zeros(T * k, I, dtype=BF16)}
    with pytest.raises(ValueError):
        layer.backward(db, s, torch.zeros(E, 2 * I, H), torch.zeros(E, H, I))


def test_the_package_has_it():
    Hp.lib()
    import moe_expert_layer_counting_gb300 as M
    from moe_expert_layer_counting_gb300 import training
    assert M.TrainableExperts is training.TrainableExperts
