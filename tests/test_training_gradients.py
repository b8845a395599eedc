"""Weights' gradients that the training objects refuse before the library is called: the first product of a backward call
already writes one of them, or adds to it (without a GPU)."""
import pytest
import torch

from tests import helpers as Hp

T, E, H, I, k = 5, 4, 64, 32, 2
BF16 = torch.bfloat16


@pytest.fixture
def training(monkeypatch):
    B = Hp.lib()
    from moe_expert_layer_counting_gb300 import training

    def called(*_, **__):
        raise AssertionError("the library was called")

    for name in ("moe_permute", "moe_grouped_forward", "moe_grouped_dgrad", "moe_grouped_wgrad", "moe_combine", "moe_gated_forward",
                 "moe_gated_dgrad"):
        monkeypatch.setattr(B, name, called)
    return training


def wrong(shape):
    """Gradients that do not fit, and whether they are to be added to."""
    good, last = torch.zeros(shape), shape[-1]
    return [(torch.zeros(shape, dtype=torch.float16), False), (torch.zeros(shape, dtype=torch.float64), True),
            (torch.zeros(*shape[:-1], last + 8), False), (torch.zeros(*shape[:-1], 2 * last)[..., ::2], False),
            (torch.zeros(*shape[:-1], 2 * last)[..., :last], True), (torch.zeros(shape, device="meta"), False),
            (torch.zeros(shape, dtype=BF16), True), (good[None], False),
            (torch.zeros(good.numel() + 1)[1:].view(shape), False)]           # 4 bytes past a multiple of 16


@pytest.mark.parametrize("case", range(9))
@pytest.mark.parametrize("which", [0, 1])
def test_experts(training, which, case):
    layer = training.TrainableExperts(torch.zeros(E, 2 * I, H, dtype=BF16), torch.zeros(E, H, I, dtype=BF16))
    s = {"row": torch.zeros(T, k, dtype=torch.int32), "token": torch.zeros(T * k, dtype=torch.int64),
         "h": torch.zeros(T * k, I, dtype=BF16), "offsets": torch.zeros(E + 1, dtype=torch.int32)}
    grads = [torch.zeros(E, 2 * I, H), torch.zeros(E, H, I)]
    grads[which], accumulate = wrong(grads[which].shape)[case]
    with pytest.raises(ValueError):
        layer.backward(torch.zeros(T, H, dtype=BF16), s, *grads, accumulate=accumulate)


@pytest.mark.parametrize("case", range(9))
@pytest.mark.parametrize("which", [0, 1])
def test_block(training, which, case):
    block = training.GatedFeedForward(torch.zeros(2 * I, H, dtype=BF16), torch.zeros(H, I, dtype=BF16))
    s = {"n": torch.zeros(T, H, dtype=BF16), "a": torch.zeros(T, 2 * I, dtype=BF16), "h": torch.zeros(T, I, dtype=BF16),
         "offsets": torch.tensor([0, T], dtype=torch.int32)}
    grads = [torch.zeros(2 * I, H), torch.zeros(H, I)]
    grads[which], accumulate = wrong(grads[which].shape)[case]
    with pytest.raises(ValueError):
        block.backward(torch.zeros(T, H, dtype=BF16), s, *grads, accumulate=accumulate)
