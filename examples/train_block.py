"""A block of the expert layer trained in BF16 and then served in FP4.

    x -> norm -> router, experts -> norm, gate, + x -> y

The block learns another block's answers: forward and backward run on the products grouped by expert and the norms
around the layer, the step is AdamW with 8-bit states over all tensors at once (float32 parameters, BF16 copies that the
products read).  Then the trained copies are cast to FP4 (``QuantizedExperts``) and the same block runs on ``MoELayer``.

    python examples/train_block.py [--steps 60] [--tokens 512] [--state-bits 8]
"""
from __future__ import annotations

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import moe_expert_layer_counting_gb300 as M  # noqa: E402
from moe_expert_layer_counting_gb300 import binding as B  # noqa: E402
from moe_expert_layer_counting_gb300.training import TrainableExperts  # noqa: E402


class Block:
    """y = x + sigmoid(gate) * norm(experts(norm(x))), gate per channel; the parameters by name in ``params``."""

    def __init__(self, E: int, H: int, I: int, k: int, seed: int, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)

        def randn(*shape, scale=1.0):
            return torch.randn(*shape, generator=g, device=device) * scale

        self.k, self.E = k, E
        self.params = {"l1": randn(E, 2 * I, H, scale=H ** -0.5), "l2": randn(E, H, I, scale=I ** -0.5),
                       "router": randn(E, H, scale=H ** -0.5), "w_pre": torch.ones(H, device=device),
                       "w_post": torch.ones(H, device=device), "gate": randn(1, H, scale=0.1)}
        self.copies = {name: p.bfloat16() for name, p in self.params.items()}

    def forward(self, x: torch.Tensor):
        """(y, what backward needs)."""
        c = self.copies
        before, after = M.BlockNorm(w_pre=c["w_pre"]), M.BlockNorm(w_post=c["w_post"], gate_sigmoid=True)
        experts = TrainableExperts(c["l1"], c["l2"])
        _, n = before.forward(x)
        logits = n.float() @ c["router"].float().T
        idx = torch.empty(x.shape[0], self.k, dtype=torch.int32, device=x.device)
        w = torch.empty(x.shape[0], self.k, device=x.device)
        B.moe_route_topk(logits, self.k, idx, w)
        b, s = experts.forward(n, idx, w)
        y, _ = after.forward(x, b, c["gate"])
        return y, (x, n, idx, w, b, y, s, before, after, experts)

    def backward(self, dy: torch.Tensor, saved) -> dict:
        """Gradients of the parameters, by name, BF16."""
        x, n, idx, w, b, y, s, before, after, experts = saved
        c = self.copies
        g = after.backward(y, b, c["gate"], dy, None)
        d = {"l1": torch.empty_like(c["l1"]), "l2": torch.empty_like(c["l2"]), "w_post": g["dw_post"], "gate": g["dgate"]}
        dn, dw = experts.backward(g["db"], s, d["l1"], d["l2"])
        # the chosen logits' softmax, then the router
        dl = torch.zeros(x.shape[0], self.E, device=x.device)
        dl.scatter_(1, idx.long(), w * (dw - (w * dw).sum(1, keepdim=True)))
        d["router"] = dl.T @ n.float()
        dn = (dn.float() + dl @ c["router"].float()).bfloat16()
        d["w_pre"] = before.backward(x, None, None, None, dn)["dw_pre"]
        assert experts.status() == B.MOE_OK
        return {name: t.bfloat16().contiguous() for name, t in d.items()}

    def serve(self, max_tokens: int):
        """The block on FP4 experts: a function of x."""
        c = self.copies
        layer = M.MoELayer(M.QuantizedExperts.from_bf16(c["l1"], c["l2"]), self.k, max_tokens)
        before, after = M.BlockNorm(w_pre=c["w_pre"]), M.BlockNorm(w_post=c["w_post"], gate_sigmoid=True)

        def run(x):
            _, n = before.forward(x)
            return after.forward(x, layer(n, n.float() @ c["router"].float().T), c["gate"])[0]

        return run


def train(steps: int, tokens: int, E=8, H=256, I=128, k=2, state_bits=8, lr=3e-3, seed=0, say=print):
    """(the block, losses): `steps` steps on the answers of another block."""
    teacher, block = Block(E, H, I, k, seed=seed + 1), Block(E, H, I, k, seed=seed + 2)
    names = list(block.params)
    opt = M.AdamW([block.params[n] for n in names], lr=lr, betas=(0.9, 0.95), weight_decay=0.0, state_bits=state_bits,
                  copies=[block.copies[n] for n in names])
    data = torch.Generator(device="cuda").manual_seed(seed + 3)
    losses = []
    for step in range(steps):
        x = torch.randn(tokens, H, generator=data, device="cuda").bfloat16()
        want, _ = teacher.forward(x)
        y, saved = block.forward(x)
        off = y.float() - want.float()
        losses.append(off.pow(2).mean())
        grads = block.backward((off * (2 / off.numel())).bfloat16(), saved)
        opt.step([grads[n] for n in names])
        if step % 10 == 0 or step == steps - 1:
            say(f"step {step}: loss {float(losses[-1]):.4f}")
    return block, [float(v) for v in losses]


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--tokens", type=int, default=512)
    ap.add_argument("--state-bits", type=int, default=8, choices=(8, 32))
    a = ap.parse_args()
    block, losses = train(a.steps, a.tokens, state_bits=a.state_bits)
    x = torch.randn(64, 256, device="cuda").bfloat16()
    y, served = block.forward(x)[0].float(), block.serve(64)(x).float()
    print(f"loss {losses[0]:.4f} -> {losses[-1]:.4f}; served in FP4, y is {float((served - y).norm() / y.norm()):.3f} off the BF16 "
          "block's")


if __name__ == "__main__":
    main()
