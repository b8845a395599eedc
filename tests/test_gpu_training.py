"""The expert layer with BF16 weights, forward and backward, and the training example that runs the new operators
together.

Tolerance of the comparison with torch's own differentiation in float64: every tensor that the layer rounds to BF16 on
the way (rows, a, h, pair rows; their gradients) carries an error of at most 2^-8 of its values, independent over the
values of a sum; no gradient passes more than six of them, so its error in norm is at most 6 * 2^-8.
"""
import importlib.util
import os

import pytest
import torch

from tests import helpers as Hp

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    Hp.lib()
    spec = importlib.util.spec_from_file_location("train_block", os.path.join(Hp.ROOT, "examples", "train_block.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("T,E,H,I,k,drop", [(1, 4, 64, 32, 1, False), (37, 8, 128, 72, 2, False), (50, 6, 136, 64, 3, True)])
def test_layer_and_gradients(example, T, E, H, I, k, drop):
    from moe_expert_layer_counting_gb300.training import TrainableExperts
    g = torch.Generator(device="cuda").manual_seed(T)

    def randn(*shape, scale=1.0):
        return torch.randn(*shape, generator=g, device="cuda") * scale

    n, l1, l2 = (t.bfloat16() for t in (randn(T, H), randn(E, 2 * I, H, scale=H ** -0.5), randn(E, H, I, scale=I ** -0.5)))
    idx = torch.stack([torch.randperm(E, generator=g, device="cuda")[:k] for _ in range(T)]).int()
    if drop:
        idx[::4, 1] = -1
        idx[7] = -1
    w, db = torch.softmax(randn(T, k), 1), randn(T, H).bfloat16()
    layer = TrainableExperts(l1, l2)
    b, s = layer.forward(n, idx, w)
    dl1, dl2 = torch.empty(E, 2 * I, H, device="cuda"), torch.empty(E, H, I, device="cuda")
    dn, dw = layer.backward(db, s, dl1, dl2)
    assert layer.status() == 0

    leaf = [t.double().requires_grad_() for t in (n, l1, l2, w)]
    out = torch.zeros(T, H, dtype=torch.float64, device="cuda")
    for j in range(k):
        e = idx[:, j].clamp(min=0).long()
        gate, up = torch.einsum("th,tih->ti", leaf[0], leaf[1][e]).split(I, 1)
        h = gate * torch.sigmoid(gate) * up * leaf[3][:, j:j + 1]
        out = out + torch.where(idx[:, j:j + 1] < 0, 0.0, torch.einsum("ti,thi->th", h, leaf[2][e]))
    grads = torch.autograd.grad((out * db.double()).sum(), leaf)
    for got, ref in ((b, out.detach()), (dn, grads[0]), (dl1, grads[1]), (dl2, grads[2]), (dw, grads[3])):
        assert float((got.double() - ref).norm()) <= 6 * 2.0 ** -8 * float(ref.norm())
    again = dl1.clone(), dl2.clone()
    layer.backward(db, s, dl1, dl2, accumulate=True)
    assert torch.allclose(dl1, 2 * again[0]) and torch.allclose(dl2, 2 * again[1])


@pytest.mark.parametrize("bits", [8, 32])
def test_training_learns_and_serves(example, bits):
    """The example's losses fall (those of its last ten steps, whatever the rate), and served in FP4 (weights with a relative step of
    up to 1/4 of a value, 1/6 of a group's largest: 0.1 to 0.2 in norm; the layer is a part of y only) the block is the
    one that was trained."""
    block, losses = example.train(steps=40, tokens=256, state_bits=bits, say=lambda *_: None)
    assert sum(losses[-10:]) < sum(losses[:10]) and all(a < losses[0] for a in losses[-10:])
    x = torch.randn(64, 256, generator=torch.Generator(device="cuda").manual_seed(9), device="cuda").bfloat16()
    y, served = block.forward(x)[0].float(), block.serve(64)(x).float()
    assert float((served - y).norm() / y.norm()) < 0.2
