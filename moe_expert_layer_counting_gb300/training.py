"""The expert layer with BF16 weights, forward and backward: what trains the weights that ``QuantizedExperts`` and
``Bfp8Experts`` are cast from.

The products, the permute and the combine are the library's; the gathers of rows and the gated activation between the
two products are plain torch operations (float32 inside, one rounding to BF16).
"""
from __future__ import annotations

import torch

from . import binding as B


class TrainableExperts:
    """b = layer(n, topk_idx, topk_w) and its gradients, with the layer's weights l1 [E, 2I, H] (gate rows then up rows)
    and l2 [E, H, I] in BF16.

    The layer is that of ``MoELayer`` without its quantisation: h = silu(gate) * up * topk_w for each (token, slot) pair,
    summed over a token's slots after the down product.  topk_idx < 0 marks a dropped pair; an index of E or more is
    reported by status() and its pair dropped.
    """

    def __init__(self, l1: torch.Tensor, l2: torch.Tensor):
        E, twoI, H = l1.shape
        if l2.shape != (E, H, twoI // 2):
            raise ValueError("l1 [E, 2I, H] and l2 [E, H, I] do not fit")
        self.l1, self.l2 = l1, l2
        self.E, self.H, self.I = E, H, twoI // 2
        dev = l1.device
        # of the products (the size does not depend on the rows) and of the last permute: status() reads each one's status
        self.workspaces = [torch.zeros(B.moe_grouped_workspace_size(1, H, 2 * self.I, E), dtype=torch.uint8, device=dev)
                           for _ in range(6)]
        self.permute_workspace = None

    def _check_rows(self, name, t, T):
        if t.shape != (T, self.H) or t.dtype is not torch.bfloat16 or t.device != self.l1.device:
            raise ValueError(f"{name} is not [{T}, {self.H}] BF16 on the weights' device")

    def _permute(self, topk_idx):
        T, k = topk_idx.shape
        dev = topk_idx.device
        counts = torch.empty(self.E, dtype=torch.int32, device=dev)
        offsets = torch.empty(self.E + 1, dtype=torch.int32, device=dev)
        perm = torch.zeros(T * k, dtype=torch.int32, device=dev)         # rows past offsets[E] belong to no expert
        inv_perm = torch.empty(T * k, dtype=torch.int32, device=dev)
        ws = torch.empty(B.moe_permute_workspace_size(T, self.E, k), dtype=torch.uint8, device=dev)
        self.permute_workspace = ws
        B.moe_permute(topk_idx, self.E, counts, offsets, perm, inv_perm, ws)
        return offsets, perm.long(), inv_perm.view(T, k)

    def _sum_slots(self, rows, s):
        """Each token's sum over its slots of its pairs' rows (float32 inside; dropped slots are left out)."""
        T, k = s["row"].shape
        by_slot = rows[s["row"].clamp(min=0).T.reshape(-1)].view(k, T, rows.shape[1])
        out = torch.empty(T, rows.shape[1], dtype=torch.bfloat16, device=rows.device)
        B.moe_combine(by_slot, s["row"], out)
        return out

    def forward(self, n: torch.Tensor, topk_idx: torch.Tensor, topk_w: torch.Tensor):
        """(b [T, H], what backward needs); n [T, H] BF16, topk_idx [T, k] int32, topk_w [T, k] float32."""
        if topk_idx.dim() != 2 or topk_idx.dtype is not torch.int32 or topk_idx.device != self.l1.device:
            raise ValueError("topk_idx is not [T, k] int32 on the weights' device")
        T, k = topk_idx.shape
        self._check_rows("n", n, T)
        if topk_w.shape != (T, k):
            raise ValueError("topk_w and topk_idx do not fit")
        offsets, perm, row = self._permute(topk_idx.contiguous())
        # row [T, k]: of each pair; -1 if it was dropped
        s = {"offsets": offsets, "row": row, "token": perm // k, "w": topk_w.reshape(-1)[perm][:, None]}
        s["rows"] = n[s["token"]]
        s["a"] = torch.zeros(T * k, 2 * self.I, dtype=torch.bfloat16, device=n.device)
        B.moe_grouped_forward(s["rows"], self.l1, offsets, s["a"], self.workspaces[0])
        gate, up = s["a"].float().split(self.I, 1)
        s["h"] = (torch.nn.functional.silu(gate) * up * s["w"]).bfloat16()
        o = torch.zeros(T * k, self.H, dtype=torch.bfloat16, device=n.device)
        B.moe_grouped_forward(s["h"], self.l2, offsets, o, self.workspaces[1])
        return self._sum_slots(o, s), s

    def backward(self, db: torch.Tensor, s: dict, dl1: torch.Tensor, dl2: torch.Tensor, accumulate: bool = False):
        """(dn [T, H], dtopk_w [T, k]); the weights' gradients go to dl1 and dl2 (BF16, or float32, then also added to)."""
        self._check_rows("db", db, s["row"].shape[0])
        do = db[s["token"]]
        dh = torch.zeros_like(s["h"])
        B.moe_grouped_dgrad(do, self.l2, s["offsets"], dh, self.workspaces[2])
        B.moe_grouped_wgrad(do, s["h"], s["offsets"], dl2, self.workspaces[3], accumulate)
        gate, up = s["a"].float().split(self.I, 1)
        sig = torch.sigmoid(gate)
        act = gate * sig
        d = dh.float()
        dw = (d * act * up).sum(1)
        d = d * s["w"]
        da = torch.cat([d * up * (sig + act * (1 - sig)), d * act], 1).bfloat16()
        drows = torch.zeros_like(s["rows"])
        B.moe_grouped_dgrad(da, self.l1, s["offsets"], drows, self.workspaces[4])
        B.moe_grouped_wgrad(da, s["rows"], s["offsets"], dl1, self.workspaces[5], accumulate)
        dtopk_w = torch.where(s["row"] < 0, 0.0, dw[s["row"].clamp(min=0)])
        return self._sum_slots(drows, s), dtopk_w

    def status(self) -> int:
        """MOE_OK, or the first status that the last step's permute or products reported (synchronises)."""
        used = self.workspaces if self.permute_workspace is None else [self.permute_workspace, *self.workspaces]
        return next((c for c in (B.moe_get_device_status(w) for w in used) if c), B.MOE_OK)
