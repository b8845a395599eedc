"""The expert layer with BF16 weights, forward and backward: what trains the weights that ``QuantizedExperts`` and
``Bfp8Experts`` are cast from.

The products, the permute and the combine are the library's; the gathers of rows are torch operations.  The gated
activation between the two products is one of the products' epilogue (``fused=True``, and ``GatedFeedForward``), or plain
torch operations between them (float32 inside, one rounding to BF16).
"""
from __future__ import annotations

import torch

from . import binding as B


def _check_gradients(dl1, dl2, l1, l2, accumulate):
    """Of a backward call, before its first product writes dl2 or adds to it."""
    kinds = (torch.float32,) if accumulate else (torch.bfloat16, torch.float32)
    for name, d, w in (("dl1", dl1, l1), ("dl2", dl2, l2)):
        if d.shape != w.shape or d.dtype not in kinds or d.device != w.device or not d.is_contiguous() or d.data_ptr() % 16:
            raise ValueError(f"{name} is not contiguous {'float32' if accumulate else 'BF16 or float32'} of the weight's shape, "
                             "on its device, aligned to 16 bytes")


class TrainableExperts:
    """b = layer(n, topk_idx, topk_w) and its gradients, with the layer's weights l1 [E, 2I, H] (gate rows then up rows)
    and l2 [E, H, I] in BF16.

    The layer is that of ``MoELayer`` without its quantisation: h = silu(gate) * up * topk_w for each (token, slot) pair,
    summed over a token's slots after the down product.  topk_idx < 0 marks a dropped pair; an index of E or more is
    reported by status() and its pair dropped.

    fused: the activation inside the products' kernels (include/moe_gated.h), which rounds less on the way: h is that of
    the unrounded gate and up values, and the gradient of h is not rounded at all.  Without it the results are those of
    separate operations, each rounded to BF16.
    """

    def __init__(self, l1: torch.Tensor, l2: torch.Tensor, fused: bool = False):
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
        self.gated_workspaces = {}                  # of the last forward and of the last backward call's gated product
        self.fused = fused

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

    def _gated_workspace(self, P):
        """A new one for each call: it holds sums, and a captured graph may write it long after the call."""
        return torch.empty(B.moe_gated_workspace_size(P, self.H, self.I, self.E), dtype=torch.uint8, device=self.l1.device)

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
        if self.fused:
            if topk_w.dtype is not torch.float32 or topk_w.device != self.l1.device:
                raise ValueError("topk_w is not float32 on the weights' device")
            h = torch.zeros(T * k, self.I, dtype=torch.bfloat16, device=n.device)
            ws = self._gated_workspace(T * k)
            B.moe_gated_forward(s["rows"], self.l1, offsets, h, ws, a=s["a"], row_w=s["w"][:, 0])
            s["h"], self.gated_workspaces["forward"] = h, ws
        else:
            B.moe_grouped_forward(s["rows"], self.l1, offsets, s["a"], self.workspaces[0])
            gate, up = s["a"].float().split(self.I, 1)
            s["h"] = (torch.nn.functional.silu(gate) * up * s["w"]).bfloat16()
        o = torch.zeros(T * k, self.H, dtype=torch.bfloat16, device=n.device)
        B.moe_grouped_forward(s["h"], self.l2, offsets, o, self.workspaces[1])
        return self._sum_slots(o, s), s

    def backward(self, db: torch.Tensor, s: dict, dl1: torch.Tensor, dl2: torch.Tensor, accumulate: bool = False):
        """(dn [T, H], dtopk_w [T, k]); the weights' gradients go to dl1 and dl2 (BF16, or float32, then also added to)."""
        self._check_rows("db", db, s["row"].shape[0])
        _check_gradients(dl1, dl2, self.l1, self.l2, accumulate)
        do = db[s["token"]]
        B.moe_grouped_wgrad(do, s["h"], s["offsets"], dl2, self.workspaces[3], accumulate)
        if self.fused:
            da = torch.zeros_like(s["a"])
            dw = torch.zeros(da.shape[0], dtype=torch.float32, device=da.device)
            ws = self._gated_workspace(da.shape[0])
            B.moe_gated_dgrad(do, self.l2, s["offsets"], s["a"], da, ws, row_w=s["w"][:, 0], drow_w=dw)
            self.gated_workspaces["backward"] = ws
        else:
            dh = torch.zeros_like(s["h"])
            B.moe_grouped_dgrad(do, self.l2, s["offsets"], dh, self.workspaces[2])
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
        """MOE_OK, or the first status that the last forward and backward call's permute and products reported (synchronises)."""
        used = ([] if self.permute_workspace is None else [self.permute_workspace]) + [*self.gated_workspaces.values()] + self.workspaces
        return next((c for c in (B.moe_get_device_status(w) for w in used) if c), B.MOE_OK)


class GatedFeedForward:
    """b = block(n), the gated feed-forward block that every token takes (a shared expert, a dense layer), and its
    gradients: h = f(n gate^T) (n up^T), b = h l2^T, with l1 [2I, H] (gate rows then up rows) and l2 [H, I] in BF16.

    activation: ACT_SILU or ACT_GELU_TANH (include/moe_gated.h).  Calls run on the current stream; each has outputs and
    workspaces of its own, of which the object keeps the last forward and the last backward call's for status().
    """

    def __init__(self, l1: torch.Tensor, l2: torch.Tensor, activation: int = B.ACT_SILU):
        if l1.dim() != 2 or l1.shape[0] % 2 or l2.shape != (l1.shape[1], l1.shape[0] // 2):
            raise ValueError("l1 [2I, H] and l2 [H, I] do not fit")
        if any(t.dtype is not torch.bfloat16 or not t.is_contiguous() for t in (l1, l2)) or l1.device != l2.device:
            raise ValueError("l1 and l2 are not contiguous BF16 on one device")
        if activation not in (B.ACT_SILU, B.ACT_GELU_TANH):
            raise ValueError("activation is ACT_SILU or ACT_GELU_TANH")
        self.l1, self.l2, self.activation = l1, l2, activation
        self.H, self.I = l1.shape[1], l2.shape[1]
        self._used = {"forward": [], "backward": []}

    def _workspaces(self, T, n):
        """One for a gated call, n - 1 for products."""
        sizes = [B.moe_gated_workspace_size(T, self.H, self.I, 1)] + [B.moe_grouped_workspace_size(T, self.H, self.I, 1)] * (n - 1)
        return [torch.empty(size, dtype=torch.uint8, device=self.l1.device) for size in sizes]

    def forward(self, n: torch.Tensor, keep: bool = True):
        """(b [T, H], what backward needs); n [T, H] BF16.  keep=False: no backward follows, and nothing is kept for it."""
        self._check(n, n.shape[0] if n.dim() == 2 else -1)
        T, new = n.shape[0], n.new_empty
        # [0, T]: all rows are the one expert's
        offsets = torch.arange(0, T + 1, max(T, 1), dtype=torch.int32, device=n.device) if T else new(2, dtype=torch.int32).zero_()
        h, b = new(T, self.I), new(T, self.H)
        a = new(T, 2 * self.I) if keep else None
        ws = self._workspaces(T, 2)
        B.moe_gated_forward(n, self.l1[None], offsets, h, ws[0], a=a, activation=self.activation)
        B.moe_grouped_forward(h, self.l2[None], offsets, b, ws[1])
        self._used["forward"] = ws
        return b, {"n": n, "a": a, "h": h, "offsets": offsets} if keep else None

    def backward(self, db: torch.Tensor, s: dict, dl1: torch.Tensor, dl2: torch.Tensor, accumulate: bool = False):
        """dn [T, H]; the weights' gradients go to dl1 and dl2 (BF16, or float32, then also added to)."""
        n, a, offsets, T = s["n"], s["a"], s["offsets"], s["n"].shape[0]
        self._check(db, T)
        _check_gradients(dl1, dl2, self.l1, self.l2, accumulate)
        da, dn = torch.empty_like(a), torch.empty_like(n, memory_format=torch.contiguous_format)
        ws = self._workspaces(T, 4)
        B.moe_grouped_wgrad(db, s["h"], offsets, dl2[None], ws[1], accumulate)
        B.moe_gated_dgrad(db, self.l2[None], offsets, a, da, ws[0], activation=self.activation)
        B.moe_grouped_dgrad(da, self.l1[None], offsets, dn, ws[2])
        B.moe_grouped_wgrad(da, n, offsets, dl1[None], ws[3], accumulate)
        self._used["backward"] = ws
        return dn

    def _check(self, t, T):
        if t.shape != (T, self.H) or t.dtype is not torch.bfloat16 or t.device != self.l1.device:
            raise ValueError(f"rows are not [T, {self.H}] BF16 on the weights' device, or not those of forward")

    def status(self) -> int:
        """MOE_OK, or the first status that the last forward and backward call's products reported (synchronises)."""
        used = self._used["forward"] + self._used["backward"]
        return next((c for c in (B.moe_get_device_status(w) for w in used) if c), B.MOE_OK)
