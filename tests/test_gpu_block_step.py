"""One training step of a block with the gated experts, a dense block, layer norm and Muon together, as they are used:

    s, n = norm(x, b);  y = experts(n) + dense(n);  loss = sum(y dy) + sum(s ds)

against float64.  Tolerance in norm: values rounded to BF16 on the way carry 2^-8 each, and no gradient passes more than
eight of them.  Muon's step is checked against the definition on the gradients that it was given, with the tolerance of
test_gpu_muon.py: experts that few rows reach have gradients of low rank, whose update carries the FP16 iterates' rounding in
the directions that they lack (0.15 in norm for rank one, as ``rounded`` says).
"""
import pytest
import torch

from tests import helpers as Hp
from tests.test_gpu_muon import orthogonal

pytestmark = pytest.mark.gpu

BF16, U = torch.bfloat16, 2.0 ** -8


@pytest.fixture(scope="module")
def M():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    Hp.lib()
    import moe_expert_layer_counting_gb300 as package
    return package


def randn(*shape, seed=0, scale=1.0, dtype=BF16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


class Block:
    """The parameters as float32 masters with BF16 copies, their gradients and the optimisers."""

    def __init__(self, M, E, H, I, shared):
        f32 = torch.float32
        self.masters = [randn(E, 2 * I, H, seed=1, scale=H ** -0.5, dtype=f32), randn(E, H, I, seed=2, scale=I ** -0.5, dtype=f32),
                        randn(2 * shared, H, seed=3, scale=H ** -0.5, dtype=f32), randn(H, shared, seed=4, scale=shared ** -0.5, dtype=f32)]
        self.copies = [p.bfloat16() for p in self.masters]
        self.norm_w = [1 + 0.1 * randn(H, seed=5, dtype=f32), 0.1 * randn(H, seed=6, dtype=f32)]
        self.grads = [torch.empty_like(p) for p in self.masters]
        self.experts = M.TrainableExperts(*self.copies[:2], fused=True)
        self.dense = M.GatedFeedForward(*self.copies[2:])
        self.norm = M.LayerNorm(*self.norm_w)
        self.muon = M.Muon(self.masters, lr=0.02, momentum=0.9, weight_decay=0.1, adjust="shape", copies=self.copies)
        self.adamw = M.AdamW(self.norm_w, lr=1e-3)

    def step(self, x, b, idx, w, dy, ds, update=True):
        s, n = self.norm.forward(x, b)
        routed, kept = self.experts.forward(n, idx, w)
        dense, kept_dense = self.dense.forward(n)
        dn, dw = self.experts.backward(dy, kept, *self.grads[:2])
        dn = dn + self.dense.backward(dy, kept_dense, *self.grads[2:])
        d = self.norm.backward(s, dn, ds)
        if update:
            self.muon.step(self.grads)
            self.adamw.step([d["dw"], d["dbias"]])
        return {"y": routed + dense, "s": s, "dx": d["dx"], "dtopk_w": dw, "dw": d["dw"], "dbias": d["dbias"]}


def inputs(T, H, E, k, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    idx = torch.stack([torch.randperm(E, generator=g, device="cuda")[:k] for _ in range(T)]).int()
    return (randn(T, H, seed=seed + 1), randn(T, H, seed=seed + 2), idx, torch.softmax(torch.randn(T, k, generator=g, device="cuda"), 1),
            randn(T, H, seed=seed + 3), randn(T, H, seed=seed + 4))


def reference(block, x, b, idx, w, dy, ds):
    """Outputs and gradients in float64, from the BF16 weights."""
    leaf = [t.double().requires_grad_() for t in (x, *block.copies, *block.norm_w, w)]
    xs, l1, l2, d1, d2, nw, nb, tw = leaf
    s = xs + b.double()
    c = s - s.mean(1, keepdim=True)
    n = c / torch.sqrt(c.square().mean(1, keepdim=True) + 1e-5) * nw + nb

    def gated(a):
        gate, up = a.chunk(2, -1)
        return gate * torch.sigmoid(gate) * up

    y = gated(n @ d1.T) @ d2.T
    for j in range(idx.shape[1]):
        e = idx[:, j].long()
        h = gated(torch.einsum("th,tih->ti", n, l1[e])) * tw[:, j:j + 1]
        y = y + torch.einsum("ti,thi->th", h, l2[e])
    loss = (y * dy.double()).sum() + (s * ds.double()).sum()
    grads = torch.autograd.grad(loss, leaf)
    return {"y": y.detach(), "s": s.detach(), "dx": grads[0], "dtopk_w": grads[7], "dw": grads[5], "dbias": grads[6]}, grads[1:5]


@pytest.mark.parametrize("T,H,I,shared,E,k", [(1, 64, 32, 40, 4, 2), (37, 136, 72, 200, 6, 2), (300, 256, 128, 264, 8, 3)])
def test_step(M, T, H, I, shared, E, k):
    block = Block(M, E, H, I, shared)
    for seed in (10, 20):                                   # the second step works on what the first wrote
        args = inputs(T, H, E, k, seed)
        want, grads = reference(block, *args)
        before, momentum = [p.double() for p in block.masters], [m.double() for m in block.muon.state["m"]]
        got = block.step(*args)
        assert block.experts.status() == 0 and block.dense.status() == 0 and block.muon.device_status() == 0
        for name, ref in want.items():
            assert float((got[name].double() - ref).norm()) <= 8 * U * float(ref.norm()), name
        for g, ref in zip(block.grads, grads):
            assert float((g.double() - ref).norm()) <= 8 * U * float(ref.norm())
        for i, p in enumerate(block.masters):
            g = block.grads[i].double()
            m = 0.9 * momentum[i] + 0.1 * g
            u = 0.9 * m + 0.1 * g
            stack = u.view(-1, *u.shape[-2:])
            o = torch.stack([orthogonal(v) for v in stack]).view_as(u)
            rate = 0.02 * max(1.0, u.shape[-2] / u.shape[-1]) ** 0.5
            ref = before[i] * (1 - 0.02 * 0.1) - rate * o
            emulated = torch.stack([orthogonal(v, rounded=True) for v in stack]).view_as(u)
            bound = 1.5 * float((emulated - o).norm()) + 1e-3 * float(o.norm())
            assert float((p.double() - ref).norm()) <= rate * bound + 2.0 ** -22 * float(ref.norm())
            assert torch.equal(block.copies[i], p.bfloat16())


def test_step_in_a_graph(M):
    """Forward and backward captured once and replayed on new inputs give the eager step's bits, with Muon's step after
    each replay."""
    T, H, I, shared, E, k = 50, 136, 72, 200, 6, 2
    eager, other = Block(M, E, H, I, shared), Block(M, E, H, I, shared)
    first, second = inputs(T, H, E, k, 10), inputs(T, H, E, k, 20)
    place = [t.clone() for t in first]
    other.step(*place, update=False)                        # what is built at the first call is built
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = other.step(*place, update=False)
    for args in (first, second):
        want = eager.step(*args, update=False)
        eager.muon.step(eager.grads)
        for p, t in zip(place, args):
            p.copy_(t)
        graph.replay()
        other.muon.step(other.grads)
        torch.cuda.synchronize()
        assert all(torch.equal(want[k], out[k]) for k in want)
        assert all(torch.equal(p, q) for p, q in zip(eager.masters, other.masters))
