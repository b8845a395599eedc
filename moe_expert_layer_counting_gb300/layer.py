"""Device-side containers around the C ABI: quantised expert weights and a
layer object that owns its workspace.  Allocation uses torch; every
computation is a call into libmoe_mxq.so."""
from __future__ import annotations

import contextlib
import itertools

import numpy as np
import torch

from . import binding as B

_TYPES = {code: kind for kind, code in B._DTYPES.items()}


def _on(stream):
    """Allocations made inside belong to `stream` (None: the current one), so that their memory is not handed on
    while work of that stream still uses it."""
    if stream is None:
        return contextlib.nullcontext()
    return torch.cuda.stream(stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(int(stream)))


class QuantizedExperts:
    """FP4 E2M1 + UE8M0 expert weights in the MMA layouts the GEMMs read.

    w1q [E, 2I, H/2] / w1s (E*2I*H/32 bytes, chunk order) -- gate/up interleaved by 8;
    w2q [E, H, I/2]  / w2s (E*H*I/32 bytes, chunk order).
    """

    def __init__(self, E: int, H: int, I: int, device="cuda"):
        self.E, self.H, self.I = E, H, I
        self.w1q = torch.empty(E, 2 * I, H // 2, dtype=torch.uint8, device=device)
        self.w1s = torch.empty(E * 2 * I * H // 32, dtype=torch.uint8, device=device)
        self.w2q = torch.empty(E, H, I // 2, dtype=torch.uint8, device=device)
        self.w2s = torch.empty(E * H * I // 32, dtype=torch.uint8, device=device)

    def set_expert(self, e: int, l1_w: torch.Tensor, l2_w: torch.Tensor, stream=None):
        """Quantise expert e from BF16 l1_w [2I, H] (gate rows then up rows) and l2_w [H, I]."""
        H, I = self.H, self.I
        assert l1_w.shape == (2 * I, H) and l2_w.shape == (H, I)
        s1 = 2 * I * H // 32
        s2 = H * I // 32
        B.mxq_quantize_weight(l1_w.contiguous().view(1, 2 * I, H), B.LAYOUT_MMA_L1, self.w1q[e],
                              self.w1s[e * s1:(e + 1) * s1], stream)
        B.mxq_quantize_weight(l2_w.contiguous().view(1, H, I), B.LAYOUT_MMA_L2, self.w2q[e],
                              self.w2s[e * s2:(e + 1) * s2], stream)

    @classmethod
    def from_bf16(cls, l1_w: torch.Tensor, l2_w: torch.Tensor, stream=None):
        E, twoI, H = l1_w.shape
        q = cls(E, H, twoI // 2, device=l1_w.device)
        B.mxq_quantize_weight(l1_w.contiguous(), B.LAYOUT_MMA_L1, q.w1q, q.w1s, stream)
        B.mxq_quantize_weight(l2_w.contiguous(), B.LAYOUT_MMA_L2, q.w2q, q.w2s, stream)
        return q


class MoELayer:
    """The MoE expert layer for a fixed (max_tokens, H, I, E, k): y = layer(x, logits)."""

    def __init__(self, weights: QuantizedExperts, k: int, max_tokens: int, tile_n: int = 0,
                 route_mode: int = B.ROUTE_SOFTMAX, schedule: int = B.SCHEDULE_DEFAULT):
        self.w = weights
        self.k = k
        self.max_tokens = max_tokens
        self.tile_n = tile_n
        self.route_mode = route_mode
        self.schedule = schedule
        nbytes = B.moe_workspace_size(max_tokens, weights.H, weights.I, weights.E, k)
        self.workspace = torch.empty(nbytes, dtype=torch.uint8, device=weights.w1q.device)

    def __call__(self, x: torch.Tensor, logits: torch.Tensor, y: torch.Tensor = None, stream=None, **outs):
        T = x.shape[0]
        assert T <= self.max_tokens
        if y is None:
            y = torch.empty_like(x)
        w = self.w
        ws = self.workspace
        need = B.moe_workspace_size(T, w.H, w.I, w.E, self.k)
        B.moe_forward(x, logits, w.w1q, w.w1s, w.w2q, w.w2s, self.k, y, ws[:need], tile_n=self.tile_n,
                      route_mode=self.route_mode, schedule=self.schedule, stream=stream, **outs)
        return y

    def device_status(self, stream=None) -> int:
        return B.moe_get_device_status(self.workspace, stream)


class Bfp8Experts:
    """Block-FP8 expert weights: E4M3 codes (tile-contiguous by default) with
    one float32 scale per 128 x 128 block.

    w1q (E*2I*H bytes) / w1s [E, 2I/128, H/128] -- gate rows [0, I), up rows [I, 2I);
    w2q (E*H*I bytes)  / w2s [E, H/128, I/128].
    """

    def __init__(self, E: int, H: int, I: int, device="cuda", layout: int = B.BFP8_LAYOUT_TILED):
        self.E, self.H, self.I, self.layout = E, H, I, layout
        self.w1q = torch.empty(E, 2 * I, H, dtype=torch.uint8, device=device)
        self.w1s = torch.empty(E, 2 * I // 128, H // 128, dtype=torch.float32, device=device)
        self.w2q = torch.empty(E, H, I, dtype=torch.uint8, device=device)
        self.w2s = torch.empty(E, H // 128, I // 128, dtype=torch.float32, device=device)

    def set_expert(self, e: int, l1_w: torch.Tensor, l2_w: torch.Tensor, stream=None):
        """Quantise expert e from BF16 l1_w [2I, H] (gate rows then up rows) and l2_w [H, I]."""
        H, I = self.H, self.I
        assert l1_w.shape == (2 * I, H) and l2_w.shape == (H, I)
        B.bfp8_quantize_weight(l1_w.contiguous().view(1, 2 * I, H), self.w1q[e:e + 1], self.w1s[e:e + 1],
                               self.layout, stream)
        B.bfp8_quantize_weight(l2_w.contiguous().view(1, H, I), self.w2q[e:e + 1], self.w2s[e:e + 1],
                               self.layout, stream)

    @classmethod
    def from_bf16(cls, l1_w: torch.Tensor, l2_w: torch.Tensor, layout: int = B.BFP8_LAYOUT_TILED, stream=None):
        E, twoI, H = l1_w.shape
        q = cls(E, H, twoI // 2, device=l1_w.device, layout=layout)
        B.bfp8_quantize_weight(l1_w.contiguous(), q.w1q, q.w1s, layout, stream)
        B.bfp8_quantize_weight(l2_w.contiguous(), q.w2q, q.w2s, layout, stream)
        return q


class MoELayerBfp8:
    """The block-FP8 MoE expert layer for a fixed (max_tokens, H, I, E, k): y = layer(x, logits)."""

    def __init__(self, weights: Bfp8Experts, k: int, max_tokens: int, route_mode: int = B.ROUTE_SOFTMAX):
        self.w = weights
        self.k = k
        self.max_tokens = max_tokens
        self.route_mode = route_mode
        nbytes = B.moe_bfp8_workspace_size(max_tokens, weights.H, weights.I, weights.E, k)
        self.workspace = torch.empty(nbytes, dtype=torch.uint8, device=weights.w1q.device)

    def __call__(self, x: torch.Tensor, logits: torch.Tensor, y: torch.Tensor = None, stream=None, **outs):
        T = x.shape[0]
        assert T <= self.max_tokens
        if y is None:
            y = torch.empty_like(x)
        w = self.w
        need = B.moe_bfp8_workspace_size(T, w.H, w.I, w.E, self.k)
        B.moe_forward_bfp8(x, logits, w.w1q, w.w1s, w.w2q, w.w2s, self.k, y, self.workspace[:need],
                           route_mode=self.route_mode, weight_layout=w.layout, stream=stream, **outs)
        return y

    def device_status(self, stream=None) -> int:
        return B.moe_get_device_status(self.workspace, stream)


class BlockNorm:
    """The norms around the layer with its gate and residual scale, forward and backward (include/moe_norm.h).

    w_post (after the layer) and w_pre (before the next one): [H] bf16 or float32, either may be None.  Each backward call
    has a workspace of its own, as a captured graph may write one long after its call; the object keeps the last of each
    stream, and the forward calls' status words, for ``device_status``.  It has to outlive the graphs captured with it.
    """

    def __init__(self, w_post: torch.Tensor = None, w_pre: torch.Tensor = None, residual_scale: float = 1.0,
                 weight_offset: float = 0.0, eps: float = 1e-6, gate_sigmoid: bool = False):
        self.w_post, self.w_pre = w_post, w_pre
        self.how = (residual_scale, weight_offset, eps, gate_sigmoid)
        self._last = {}                             # (device, stream handle) -> workspace of the last backward call
        self._status = {}                           # the same -> status words of its forward calls

    def forward(self, x: torch.Tensor, b: torch.Tensor = None, gate: torch.Tensor = None, stream=None):
        """(y, n): the stream after the layer and the next layer's input.  Without b: (x, norm of x).  Without w_pre: n None."""
        if stream is not None:
            with _on(stream):
                return self._forward(x, b, gate, stream)
        return self._forward(x, b, gate, None)

    def _forward(self, x, b, gate, stream):
        if b is None and gate is None and self.w_pre is None:
            return x, None                          # nothing to compute
        flat = torch.contiguous_format
        y = torch.empty_like(x, memory_format=flat) if b is not None else None
        n = None
        if self.w_pre is not None:
            n = torch.empty_like(x if b is None else b, dtype=torch.bfloat16, memory_format=flat)
        handle = B._stream(stream)
        key = x.get_device(), handle
        status = self._status.get(key)
        if status is None:
            status = self._status[key] = x.new_empty(64, dtype=torch.uint8)
        B.moe_norm_forward(x, b, gate, self.w_post if b is not None else None, self.w_pre, y, n, *self.how, handle, status=status)
        return (x if y is None else y), n

    def backward(self, y: torch.Tensor, b: torch.Tensor, gate: torch.Tensor, dy: torch.Tensor, dn: torch.Tensor,
                 stream=None) -> dict:
        """Gradients dx, db, dgate, dw_post, dw_pre (None where there is nothing to differentiate) from those of
        forward's y and n (either may be None); y, b and gate are what forward returned and took.  Without b and dn, dx is dy."""
        if stream is not None:
            with _on(stream):
                return self._backward(y, b, gate, dy, dn, stream)
        return self._backward(y, b, gate, dy, dn, None)

    def _backward(self, y, b, gate, dy, dn, stream):
        if b is None and gate is None and dn is None:
            dx = torch.zeros_like(y) if dy is None else dy
            return {"dx": dx, "db": None, "dgate": None, "dw_post": None, "dw_pre": None}
        new, flat = torch.empty_like, torch.contiguous_format
        w_post = self.w_post if b is not None else None
        w_pre = self.w_pre if dn is not None else None
        dx = new(y, memory_format=flat)
        db = None if b is None else new(b, memory_format=flat)
        dgate = None if gate is None else new(gate, memory_format=flat)
        dw_post = None if w_post is None else new(w_post, dtype=torch.float32)
        dw_pre = None if w_pre is None else new(w_pre, dtype=torch.float32)
        handle = B._stream(stream)
        key = y.get_device(), handle
        self._last.pop(key, None)                   # before the next one, which may be the same memory
        ws = self._last[key] = y.new_empty(B.moe_norm_workspace_size(*y.shape), dtype=torch.uint8)
        B.moe_norm_backward(y, b, gate, w_post, w_pre, dy, dn, ws, dx, db, dgate, dw_post, dw_pre, *self.how, handle)
        return {"dx": dx, "db": db, "dgate": dgate, "dw_post": dw_post, "dw_pre": dw_pre}

    def device_status(self, stream=None) -> int:
        """MOE_OK, or what the last backward or else the last forward call on this stream reported (synchronises)."""
        key = torch.cuda.current_device(), B._stream(stream)
        words = [w for w in (self._last.get(key), self._status.get(key)) if w is not None]
        return next((code for code in (B.moe_get_device_status(w, stream) for w in words) if code), B.MOE_OK)


def _capturing(stream) -> bool:
    if not torch.cuda.is_initialized():
        return False
    if stream is None:
        return torch.cuda.is_current_stream_capturing()
    with _on(stream):
        return torch.cuda.is_current_stream_capturing()


class AdamW:
    """AdamW over a list of tensors, all updated by one call (include/moe_adamw.h).

    params: contiguous, all bf16 or all float32.  copies: a bf16 copy of each float32 parameter, written by every step
    (what the next forward pass reads).  state_bits 32: float32 states m, v; 8: E4M3 codes m, v (of sqrt v) with one
    UE8M0 byte per 32 values, m_scale, v_scale.  step and state resume a run: the steps taken so far and the lists
    (m, v) or (m, v, m_scale, v_scale) as an earlier object's ``state``; they are used in place.

    A step updates the tensors that ``params``, ``state`` and ``copies`` hold then, where their values lie then
    (``p.data = ...`` or another tensor in a list); sizes and types stay.  The storages that a step worked on are kept until
    one finds others in their place.  A step is not for capture into a graph: its number
    and rate are part of the launch, and every replay would be the same step.
    """

    def __init__(self, params, lr: float = 1e-3, betas=(0.9, 0.999), eps: float = 1e-8, weight_decay: float = 1e-2,
                 state_bits: int = 32, copies=None, step: int = 0, state=None):
        self.params, self.copies = list(params), None if copies is None else list(copies)
        self.lr, self.betas, self.eps, self.weight_decay = lr, betas, eps, weight_decay
        self.state_bits, self.steps = state_bits, step
        if state_bits not in (32, 8):
            raise ValueError("state_bits is 32 or 8")
        p_kind = self.params[0].dtype if self.params else torch.float32
        if p_kind not in B._DTYPES or any(p.dtype is not p_kind for p in self.params):
            raise ValueError("parameters are all bf16 or all float32")
        self.p_dtype = B._DTYPES[p_kind]
        if state is None:
            kind = torch.float32 if state_bits == 32 else torch.uint8
            m, v = ([torch.zeros(p.numel(), dtype=kind, device=p.device) for p in self.params] for _ in range(2))
            scales = ([torch.zeros(-(-p.numel() // 32), dtype=torch.uint8, device=p.device) for p in self.params]
                      for _ in range(2)) if state_bits == 8 else (None, None)
            state = (m, v, *scales)
        names = ("m", "v", "m_scale", "v_scale") if state_bits == 8 else ("m", "v")
        self.state = {k: list(s) for k, s in zip(names, state)}
        self.table = np.zeros(len(self.params), B.ADAMW_TENSOR)
        self.table["n"] = self.sizes = [p.numel() for p in self.params]
        self._look_up()

    def _lists(self):
        """(name of the table's column, tensors) of everything but the gradients."""
        return [("p", self.params), *self.state.items()] + ([] if self.copies is None else [("copy", self.copies)])

    def _look_up(self):
        """Checks all tensors but the gradients and puts their addresses into the table.

        Their storages are kept, so that no other can come to lie at an address in the table: while the tensors'
        addresses are those, the table is theirs.
        """
        self._seen, seen, kept = None, [], []
        for name, tensors in self._lists():
            kind = {"p": _TYPES[self.p_dtype], "copy": torch.bfloat16}.get(
                name, torch.float32 if self.state_bits == 32 else torch.uint8)
            sizes = [-(-n // 32) for n in self.sizes] if name.endswith("scale") else self.sizes
            if len(tensors) != len(sizes) or [t.numel() for t in tensors if t.dtype is kind and t.is_contiguous()] != sizes:
                raise ValueError(f"{name}: sizes, types or strides do not fit the parameters")
            kept += [t.untyped_storage() for t in tensors]
            self.table[name] = at = [t.data_ptr() for t in tensors]
            seen += at
        self._kept, self._seen, self._address = kept, seen, self.table.ctypes.data

    def __getstate__(self):
        """A copy (copy, pickle) has a table and tensors of its own, at addresses that its first step looks up."""
        return {**self.__dict__, "table": self.table.copy(), "_kept": None, "_seen": None, "_address": None}

    def step(self, grads, grad_scale: torch.Tensor = None, stream=None):
        """One step with these gradients (contiguous, all bf16 or all float32), each times grad_scale (a device float)."""
        if _capturing(stream):
            raise RuntimeError("AdamW.step in a graph's capture: every replay would be the same step")
        kind = grads[0].dtype if grads else torch.float32
        if kind not in B._DTYPES or [g.numel() for g in grads if g.dtype is kind and g.is_contiguous()] != self.sizes:
            raise ValueError("gradients: sizes, types or strides do not fit the parameters")
        # a look at every address (19 parameters: 5 us) instead of at all that _look_up checks (25 us)
        if [*map(torch.Tensor.data_ptr, itertools.chain(*(tensors for _, tensors in self._lists())))] != self._seen:
            self._look_up()
        self.table["g"] = [g.data_ptr() for g in grads]
        B.moe_adamw_step(self.table, self.p_dtype, B._DTYPES[kind], self.state_bits, self.lr, *self.betas, self.eps,
                         self.weight_decay, self.steps + 1, grad_scale, stream=stream, address=self._address)
        self.steps += 1
