"""ctypes binding of libmoe_mxq.so -- argument marshalling only.

Every function has the name of the C entry point it calls (include/moe_mxq.h,
include/moe_bfp8.h, include/moe_grouped.h,
include/moe_norm.h, include/moe_adamw.h) and takes torch tensors for the device buffers; all work runs in the
library's CUDA kernels on the given (default: current) stream.  PyTorch is
used for device memory and streams only.  A non-zero status raises MoeError.
There is no CPU fallback: importing this module without the built library
raises.
"""
from __future__ import annotations

import ctypes
import os
import struct

import numpy as np
import torch

# MOE_MXQ_LIB may point at another build of the same library (e.g. one built
# with -DMOE_MXQ_WAIT_STATS for wait-time accounting).
_LIB_PATH = os.environ.get("MOE_MXQ_LIB") or os.path.join(os.path.dirname(os.path.abspath(__file__)),
                                                          "libmoe_mxq.so")

if not os.path.exists(_LIB_PATH):
    raise ImportError(
        f"{_LIB_PATH} is missing: build it with `python -c 'import __graft_entry__ as g; g.build()'` "
        "or `python moe_expert_layer_counting_gb300/build.py`")

lib = ctypes.CDLL(_LIB_PATH)

_i64, _i32, _sz, _p = ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t, ctypes.c_void_p

MOE_OK = 0
MOE_ERR_INVALID_ARG = 1
MOE_ERR_UNSUPPORTED_SHAPE = 2
MOE_ERR_MISALIGNED = 3
MOE_ERR_WORKSPACE_TOO_SMALL = 4
MOE_ERR_CUDA = 5
MOE_ERR_TIMEOUT = 6
MOE_ERR_DEVICE_INDEX = 7

LAYOUT_CANONICAL, LAYOUT_MMA_L1, LAYOUT_MMA_L2 = 0, 1, 2
PHASE_TOKEN_SCALES, PHASE_GEMM1, PHASE_GEMM2, PHASE_H_SCALES, PHASE_RESET = 1, 2, 4, 8, 16
SCHEDULE_DEFAULT, SCHEDULE_SEPARATE, SCHEDULE_EXPERT_WAVES = 0, 1, 2
ROUTE_SOFTMAX, ROUTE_SIGMOID, ROUTE_RAW, ROUTE_NO_RENORM = 0, 1, 2, 4
BFP8_LAYOUT_CANONICAL, BFP8_LAYOUT_TILED = 0, 1
BF16, F32 = 0, 1                                         # enum moe_dtype
_DTYPES = {torch.bfloat16: BF16, torch.float32: F32}
GATE_NONE, GATE_TOKEN, GATE_CHANNEL, GATE_FULL = 0, 1, 2, 3

EXPORTED = ["mxq_quantize_act", "mxq_quantize_weight", "moe_route_topk", "moe_route_topk_ex",
            "moe_permute_workspace_size",
            "moe_permute", "moe_permute_noalloc", "moe_expert_workspace_size", "moe_expert_forward", "moe_combine",
            "moe_workspace_size", "moe_forward", "moe_get_device_status", "moe_status_string", "moe_version",
            "bfp8_quantize_act", "bfp8_quantize_weight", "moe_bfp8_workspace_size", "moe_forward_bfp8",
            "moe_grouped_workspace_size", "moe_grouped_forward", "moe_grouped_dgrad", "moe_grouped_wgrad",
            "moe_norm_forward", "moe_norm_workspace_size", "moe_norm_backward", "moe_adamw_step"]


class MoeExpertArgs(ctypes.Structure):
    _fields_ = [("struct_size", ctypes.c_uint32),
                ("T", _i64), ("H", _i64), ("I", _i64),
                ("E", _i32), ("k", _i32),
                ("xq", _p), ("xs", _p),
                ("w1q", _p), ("w1s", _p), ("w2q", _p), ("w2s", _p),
                ("topk_idx", _p), ("topk_w", _p),
                ("counts", _p), ("offsets", _p), ("perm", _p),
                ("y_pairs", _p), ("hq", _p), ("hs", _p),
                ("tile_n", _i32), ("phases", _i32),
                ("workspace", _p), ("workspace_bytes", _sz)]


class MoeForwardArgs(ctypes.Structure):
    _fields_ = [("struct_size", ctypes.c_uint32),
                ("T", _i64), ("H", _i64), ("I", _i64),
                ("E", _i32), ("k", _i32),
                ("x", _p), ("logits", _p),
                ("w1q", _p), ("w1s", _p), ("w2q", _p), ("w2s", _p),
                ("y", _p),
                ("topk_idx_out", _p), ("topk_w_out", _p),
                ("counts_out", _p), ("offsets_out", _p), ("perm_out", _p),
                ("tile_n", _i32),
                ("workspace", _p), ("workspace_bytes", _sz),
                ("route_mode", _i32), ("phases", _i32), ("schedule", _i32)]


class MoeBfp8Args(ctypes.Structure):
    _fields_ = [("struct_size", ctypes.c_uint32),
                ("T", _i64), ("H", _i64), ("I", _i64),
                ("E", _i32), ("k", _i32), ("route_mode", _i32),
                ("x", _p), ("logits", _p), ("w1q", _p), ("w1s", _p), ("w2q", _p), ("w2s", _p), ("y", _p),
                ("topk_idx_out", _p), ("topk_w_out", _p), ("counts_out", _p), ("offsets_out", _p),
                ("perm_out", _p), ("hq_out", _p), ("hs_out", _p),
                ("workspace", _p), ("workspace_bytes", _sz), ("weight_layout", _i32), ("phases", _i32)]


class MoeNormArgs(ctypes.Structure):
    _fields_ = [("struct_size", ctypes.c_uint32),
                ("x_dtype", _i32), ("w_dtype", _i32), ("gate_dtype", _i32), ("gate_kind", _i32), ("gate_sigmoid", _i32),
                ("residual_scale", ctypes.c_float), ("weight_offset", ctypes.c_float), ("eps", ctypes.c_float),
                ("T", _i64), ("H", _i64), ("x", _p), ("ldx", _i64), ("b", _p), ("ldb", _i64),
                ("gate", _p), ("ld_gate", _i64), ("w_post", _p), ("w_pre", _p),
                ("y", _p), ("ldy", _i64), ("n", _p), ("ldn", _i64), ("status", _p)]


class MoeNormGrads(ctypes.Structure):
    _fields_ = [("struct_size", ctypes.c_uint32),
                ("dy", _p), ("ld_dy", _i64), ("dn", _p), ("ld_dn", _i64), ("dx", _p), ("ld_dx", _i64),
                ("db", _p), ("ld_db", _i64), ("dgate", _p), ("ld_dgate", _i64), ("dw_post", _p), ("dw_pre", _p),
                ("workspace", _p), ("workspace_bytes", _sz)]


# moe_adamw_tensor, for host tables (numpy structured arrays)
ADAMW_TENSOR = np.dtype([(f, np.int64) for f in ("n", "p", "g", "m", "v", "m_scale", "v_scale", "copy")])


class MoeAdamwArgs(ctypes.Structure):
    _fields_ = [("struct_size", ctypes.c_uint32), ("n_tensors", _i32), ("tensors", _p),
                ("p_dtype", _i32), ("g_dtype", _i32), ("state_bits", _i32), ("grad_scale", _p),
                ("lr", ctypes.c_double), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double), ("eps", ctypes.c_double),
                ("weight_decay", ctypes.c_double), ("step", _i64)]


lib.mxq_quantize_act.argtypes = [_p, _i64, _i64, _p, _p, _p]
lib.mxq_quantize_weight.argtypes = [_p, _i64, _i64, _i64, ctypes.c_int, _p, _p, _p]
lib.moe_route_topk.argtypes = [_p, _i64, _i32, _i32, _p, _p, _p]
lib.moe_route_topk_ex.argtypes = [_p, _i64, _i32, _i32, _i32, _p, _p, _p]
lib.moe_permute_workspace_size.argtypes = [_i64, _i32, _i32]
lib.moe_permute_workspace_size.restype = _sz
lib.moe_permute.argtypes = [_p, _i64, _i32, _i32, _p, _p, _p, _p, _p, _sz, _p]
lib.moe_permute_noalloc.argtypes = [_p, _i64, _i32, _i32, _p, _p, _p, _p, _p, _p]
lib.moe_expert_workspace_size.argtypes = [_i64, _i64, _i64, _i32, _i32]
lib.moe_expert_workspace_size.restype = _sz
lib.moe_expert_forward.argtypes = [ctypes.POINTER(MoeExpertArgs), _p]
lib.moe_combine.argtypes = [_p, _p, _i64, _i32, _i64, _p, _p]
lib.moe_workspace_size.argtypes = [_i64, _i64, _i64, _i32, _i32]
lib.moe_workspace_size.restype = _sz
lib.moe_forward.argtypes = [ctypes.POINTER(MoeForwardArgs), _p]
lib.bfp8_quantize_act.argtypes = [_p, _i64, _i64, _p, _p, _p]
lib.bfp8_quantize_weight.argtypes = [_p, _i64, _i64, _i64, ctypes.c_int, _p, _p, _p]
lib.moe_bfp8_workspace_size.argtypes = [_i64, _i64, _i64, _i32, _i32]
lib.moe_bfp8_workspace_size.restype = _sz
lib.moe_forward_bfp8.argtypes = [ctypes.POINTER(MoeBfp8Args), _p]
lib.moe_grouped_workspace_size.argtypes = [_i64, _i64, _i64, _i32]
lib.moe_grouped_workspace_size.restype = _sz
lib.moe_grouped_forward.argtypes = [_p, _i64, _p, _p, _i64, _i64, _i64, _i32, _p, _i64, _p, _sz, _p]
lib.moe_grouped_dgrad.argtypes = lib.moe_grouped_forward.argtypes
lib.moe_grouped_wgrad.argtypes = [_p, _i64, _p, _i64, _p, _i64, _i64, _i64, _i32, _p, _i32, _i32, _p, _sz, _p]
lib.moe_norm_forward.argtypes = [_p, _p]                # packed structures (below) or byref of the ctypes ones
lib.moe_norm_workspace_size.argtypes = [_i64, _i64]
lib.moe_norm_workspace_size.restype = _sz
lib.moe_norm_backward.argtypes = [_p, _p, _p]
lib.moe_adamw_step.argtypes = [_p, _p]
lib.moe_get_device_status.argtypes = [_p, _p, ctypes.POINTER(ctypes.c_int)]
lib.moe_status_string.argtypes = [ctypes.c_int]
lib.moe_status_string.restype = ctypes.c_char_p
lib.moe_version.restype = ctypes.c_char_p
for _name in ("mxq_quantize_act", "mxq_quantize_weight", "moe_route_topk", "moe_route_topk_ex", "moe_permute",
              "moe_permute_noalloc",
              "moe_expert_forward",
              "moe_combine", "moe_forward", "moe_get_device_status", "bfp8_quantize_act", "bfp8_quantize_weight",
              "moe_forward_bfp8", "moe_grouped_forward", "moe_grouped_dgrad", "moe_grouped_wgrad",
              "moe_norm_forward", "moe_norm_backward", "moe_adamw_step"):
    getattr(lib, _name).restype = ctypes.c_int


class MoeError(RuntimeError):
    def __init__(self, code: int, where: str):
        super().__init__(f"{where}: {moe_status_string(code)} (status {code})")
        self.code = code


def moe_status_string(code: int) -> str:
    return lib.moe_status_string(int(code)).decode()


def moe_version() -> str:
    return lib.moe_version().decode()


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    """The stream's handle; None: the current stream (asked for without making a torch.cuda.Stream, which costs 3 us)."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _check(rc: int, where: str):
    if rc != MOE_OK:
        raise MoeError(rc, where)


def mxq_quantize_act(x: torch.Tensor, q: torch.Tensor, s: torch.Tensor, stream=None, check=True) -> int:
    """x bf16 [rows, K] -> q uint8 [rows, K] (E4M3), s uint8 [rows, K/32] (UE8M0)."""
    rows, K = x.shape
    rc = lib.mxq_quantize_act(_ptr(x), rows, K, _ptr(q), _ptr(s), _stream(stream))
    if check:
        _check(rc, "mxq_quantize_act")
    return rc


def mxq_quantize_weight(w: torch.Tensor, layout: int, q: torch.Tensor, s: torch.Tensor, stream=None,
                        check=True) -> int:
    """w bf16 [G, N, K] -> q uint8 [G, N, K/2] (packed E2M1), s uint8 (G*N*K/32 bytes)."""
    G, N, K = w.shape
    rc = lib.mxq_quantize_weight(_ptr(w), G, N, K, layout, _ptr(q), _ptr(s), _stream(stream))
    if check:
        _check(rc, "mxq_quantize_weight")
    return rc


def moe_route_topk(logits: torch.Tensor, k: int, topk_idx: torch.Tensor, topk_w: torch.Tensor, stream=None,
                   check=True, mode: int = ROUTE_SOFTMAX) -> int:
    T, E = logits.shape
    if mode == ROUTE_SOFTMAX:
        rc = lib.moe_route_topk(_ptr(logits), T, E, k, _ptr(topk_idx), _ptr(topk_w), _stream(stream))
    else:
        rc = lib.moe_route_topk_ex(_ptr(logits), T, E, k, mode, _ptr(topk_idx), _ptr(topk_w), _stream(stream))
    if check:
        _check(rc, "moe_route_topk")
    return rc


def moe_permute_workspace_size(T: int, E: int, k: int) -> int:
    return int(lib.moe_permute_workspace_size(T, E, k))


def moe_permute(topk_idx: torch.Tensor, E: int, counts, offsets, perm, inv_perm, workspace: torch.Tensor,
                stream=None, check=True) -> int:
    T, k = topk_idx.shape
    rc = lib.moe_permute(_ptr(topk_idx), T, E, k, _ptr(counts), _ptr(offsets), _ptr(perm), _ptr(inv_perm),
                         _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream))
    if check:
        _check(rc, "moe_permute")
    return rc


def moe_permute_noalloc(topk_idx: torch.Tensor, E: int, counts, offsets, perm, inv_perm, device_status=None,
                        stream=None, check=True) -> int:
    """moe_permute without a workspace: the scratch is the library's own
    device array (see include/moe_mxq.h for the size limit and sharing rules)."""
    T, k = topk_idx.shape
    rc = lib.moe_permute_noalloc(_ptr(topk_idx), T, E, k, _ptr(counts), _ptr(offsets), _ptr(perm),
                                 _ptr(inv_perm), _ptr(device_status), _stream(stream))
    if check:
        _check(rc, "moe_permute_noalloc")
    return rc


def moe_expert_workspace_size(T: int, H: int, I: int, E: int, k: int) -> int:
    return int(lib.moe_expert_workspace_size(T, H, I, E, k))


def moe_expert_forward(xq, xs, w1q, w1s, w2q, w2s, topk_idx, topk_w, counts, offsets, perm, y_pairs,
                       workspace, hq=None, hs=None, tile_n: int = 0, phases: int = 0, stream=None,
                       check=True) -> int:
    T, H = xq.shape
    E = w1q.shape[0]
    I = w2q.shape[2] * 2
    k = topk_idx.shape[1]
    a = MoeExpertArgs(ctypes.sizeof(MoeExpertArgs), T, H, I, E, k,
                      _ptr(xq), _ptr(xs), _ptr(w1q), _ptr(w1s), _ptr(w2q), _ptr(w2s),
                      _ptr(topk_idx), _ptr(topk_w), _ptr(counts), _ptr(offsets), _ptr(perm),
                      _ptr(y_pairs), _ptr(hq), _ptr(hs), tile_n, phases,
                      _ptr(workspace), workspace.numel() * workspace.element_size())
    rc = lib.moe_expert_forward(ctypes.byref(a), _stream(stream))
    if check:
        _check(rc, "moe_expert_forward")
    return rc


def moe_combine(y_pairs: torch.Tensor, topk_idx: torch.Tensor, y: torch.Tensor, stream=None, check=True) -> int:
    k, T, H = y_pairs.shape
    rc = lib.moe_combine(_ptr(y_pairs), _ptr(topk_idx), T, k, H, _ptr(y), _stream(stream))
    if check:
        _check(rc, "moe_combine")
    return rc


def moe_workspace_size(T: int, H: int, I: int, E: int, k: int) -> int:
    return int(lib.moe_workspace_size(T, H, I, E, k))


def moe_forward(x, logits, w1q, w1s, w2q, w2s, k: int, y, workspace, topk_idx_out=None, topk_w_out=None,
                counts_out=None, offsets_out=None, perm_out=None, tile_n: int = 0, stream=None, check=True,
                route_mode: int = ROUTE_SOFTMAX, phases: int = 0, schedule: int = 0) -> int:
    T, H = x.shape
    E = logits.shape[1]
    I = w2q.shape[2] * 2
    a = MoeForwardArgs(ctypes.sizeof(MoeForwardArgs), T, H, I, E, k,
                       _ptr(x), _ptr(logits), _ptr(w1q), _ptr(w1s), _ptr(w2q), _ptr(w2s), _ptr(y),
                       _ptr(topk_idx_out), _ptr(topk_w_out), _ptr(counts_out), _ptr(offsets_out),
                       _ptr(perm_out), tile_n, _ptr(workspace), workspace.numel() * workspace.element_size(),
                       route_mode, phases, schedule)
    rc = lib.moe_forward(ctypes.byref(a), _stream(stream))
    if check:
        _check(rc, "moe_forward")
    return rc


def moe_get_device_status(workspace: torch.Tensor, stream=None) -> int:
    out = ctypes.c_int(0)
    _check(lib.moe_get_device_status(_ptr(workspace), _stream(stream), ctypes.byref(out)),
           "moe_get_device_status")
    return int(out.value)


# ---------------------------------------------------------------- block-FP8 variant (include/moe_bfp8.h)

def bfp8_quantize_act(x: torch.Tensor, q: torch.Tensor, s: torch.Tensor, stream=None, check=True) -> int:
    """x bf16 [rows, K] -> q uint8 [rows, K] (E4M3), s float32 [rows, K/128]."""
    rows, K = x.shape
    rc = lib.bfp8_quantize_act(_ptr(x), rows, K, _ptr(q), _ptr(s), _stream(stream))
    if check:
        _check(rc, "bfp8_quantize_act")
    return rc


def bfp8_quantize_weight(w: torch.Tensor, q: torch.Tensor, s: torch.Tensor, layout: int = BFP8_LAYOUT_TILED,
                         stream=None, check=True) -> int:
    """w bf16 [G, N, K] -> q uint8 (E4M3, G*N*K codes in ``layout``), s float32 [G, N/128, K/128]."""
    G, N, K = w.shape
    rc = lib.bfp8_quantize_weight(_ptr(w), G, N, K, layout, _ptr(q), _ptr(s), _stream(stream))
    if check:
        _check(rc, "bfp8_quantize_weight")
    return rc


def moe_bfp8_workspace_size(T: int, H: int, I: int, E: int, k: int) -> int:
    return int(lib.moe_bfp8_workspace_size(T, H, I, E, k))


def moe_forward_bfp8(x, logits, w1q, w1s, w2q, w2s, k: int, y, workspace, topk_idx_out=None, topk_w_out=None,
                     counts_out=None, offsets_out=None, perm_out=None, hq_out=None, hs_out=None,
                     route_mode: int = ROUTE_SOFTMAX, phases: int = 0, weight_layout: int = BFP8_LAYOUT_TILED,
                     stream=None, check=True) -> int:
    T, H = x.shape
    E = logits.shape[1]
    I = w2s.shape[2] * 128
    a = MoeBfp8Args(ctypes.sizeof(MoeBfp8Args), T, H, I, E, k, route_mode,
                    _ptr(x), _ptr(logits), _ptr(w1q), _ptr(w1s), _ptr(w2q), _ptr(w2s), _ptr(y),
                    _ptr(topk_idx_out), _ptr(topk_w_out), _ptr(counts_out), _ptr(offsets_out), _ptr(perm_out),
                    _ptr(hq_out), _ptr(hs_out), _ptr(workspace), workspace.numel() * workspace.element_size(),
                    weight_layout, phases)
    rc = lib.moe_forward_bfp8(ctypes.byref(a), _stream(stream))
    if check:
        _check(rc, "moe_forward_bfp8")
    return rc


# ---------------------------------------------------------------- BF16 products grouped by expert (include/moe_grouped.h)

def _invalid(where: str, check: bool) -> int:
    if check:
        raise MoeError(MOE_ERR_INVALID_ARG, where)
    return MOE_ERR_INVALID_ARG


def _rows(t: torch.Tensor, shape: tuple, dtype=torch.bfloat16):
    """(pointer, row stride) of a tensor of this shape and type whose rows are contiguous; None if it is not."""
    if t.dtype is not dtype or t.shape != shape:
        return None
    if t.is_contiguous():
        return t.data_ptr(), shape[1]
    return (t.data_ptr(), t.stride(0)) if t.stride(1) == 1 else None


def _is_offsets(t: torch.Tensor, E: int) -> bool:
    return t.dtype is torch.int32 and t.shape == (E + 1,) and t.is_contiguous()


def moe_grouped_workspace_size(P: int, N: int, K: int, E: int) -> int:
    return int(lib.moe_grouped_workspace_size(P, N, K, E))


def _is_weight(t: torch.Tensor) -> bool:
    return t.dtype is torch.bfloat16 and t.is_contiguous()


def moe_grouped_forward(x: torch.Tensor, w: torch.Tensor, offsets: torch.Tensor, y: torch.Tensor,
                        workspace: torch.Tensor, stream=None, check=True) -> int:
    """y [P, N] = x [P, K] @ w[e] [N, K]^T for the rows offsets[e] .. offsets[e+1] of expert e (all bf16)."""
    E, N, K = w.shape
    P = x.shape[0]
    xr, yr = _rows(x, (P, K)), _rows(y, (P, N))
    if xr is None or yr is None or not _is_weight(w) or not _is_offsets(offsets, E):
        return _invalid("moe_grouped_forward", check)
    rc = lib.moe_grouped_forward(*xr, w.data_ptr(), offsets.data_ptr(), P, N, K, E, *yr, workspace.data_ptr(),
                                 workspace.nbytes, _stream(stream))
    if check:
        _check(rc, "moe_grouped_forward")
    return rc


def moe_grouped_dgrad(dy: torch.Tensor, w: torch.Tensor, offsets: torch.Tensor, dx: torch.Tensor,
                      workspace: torch.Tensor, stream=None, check=True) -> int:
    """dx [P, K] = dy [P, N] @ w[e] [N, K] for the rows offsets[e] .. offsets[e+1] of expert e (all bf16)."""
    E, N, K = w.shape
    P = dy.shape[0]
    yr, xr = _rows(dy, (P, N)), _rows(dx, (P, K))
    if xr is None or yr is None or not _is_weight(w) or not _is_offsets(offsets, E):
        return _invalid("moe_grouped_dgrad", check)
    rc = lib.moe_grouped_dgrad(*yr, w.data_ptr(), offsets.data_ptr(), P, N, K, E, *xr, workspace.data_ptr(),
                               workspace.nbytes, _stream(stream))
    if check:
        _check(rc, "moe_grouped_dgrad")
    return rc


def moe_grouped_wgrad(dy: torch.Tensor, x: torch.Tensor, offsets: torch.Tensor, dw: torch.Tensor,
                      workspace: torch.Tensor, accumulate: bool = False, stream=None, check=True) -> int:
    """dw [E, N, K] (bf16 or float32) = dy[rows of e]^T @ x[rows of e]; accumulate adds to a float32 dw."""
    E, N, K = dw.shape
    P = dy.shape[0]
    yr, xr, kind = _rows(dy, (P, N)), _rows(x, (P, K)), _DTYPES.get(dw.dtype)
    if xr is None or yr is None or kind is None or not dw.is_contiguous() or not _is_offsets(offsets, E):
        return _invalid("moe_grouped_wgrad", check)
    rc = lib.moe_grouped_wgrad(*yr, *xr, offsets.data_ptr(), P, N, K, E, dw.data_ptr(), kind, 1 if accumulate else 0,
                               workspace.data_ptr(), workspace.nbytes, _stream(stream))
    if check:
        _check(rc, "moe_grouped_wgrad")
    return rc


# ---------------------------------------------------------------- norms around the layer (include/moe_norm.h)

# MoeNormArgs, MoeNormGrads and MoeAdamwArgs as bytes: packing costs a fifth of filling a ctypes structure
_NORM_ARGS = struct.Struct("@I5i3fqqPqPqPqPPPqPqP")
_NORM_GRADS = struct.Struct("@IPqPqPqPqPqPPPN")
_ADAMW_ARGS = struct.Struct("@IiPiiiP5dq")
assert (_NORM_ARGS.size, _NORM_GRADS.size, _ADAMW_ARGS.size) == tuple(
    ctypes.sizeof(c) for c in (MoeNormArgs, MoeNormGrads, MoeAdamwArgs))
_NONE = (0, 0)


def _norm_args(x, b, gate, w_post, w_pre, y, n, residual_scale, weight_offset, eps, gate_sigmoid, status=0):
    """The bytes of MoeNormArgs for these tensors, or None if a type, shape or stride does not fit."""
    shape = T, H = x.shape
    dtype = x.dtype
    xt = _DTYPES.get(dtype)
    xr = _rows(x, shape, dtype)
    br = _NONE if b is None else _rows(b, shape)
    yr = _NONE if y is None else _rows(y, shape, dtype)
    nr = _NONE if n is None else _rows(n, shape)
    if xt is None or xr is None or br is None or yr is None or nr is None:
        return None
    wt, post, pre, kinds = BF16, 0, 0, None
    if w_pre is not None:
        kinds, pre = w_pre.dtype, w_pre.data_ptr()
        wt = _DTYPES.get(kinds)
        if wt is None or w_pre.shape != (H,) or not w_pre.is_contiguous():
            return None
    if w_post is not None:
        kind, post = w_post.dtype, w_post.data_ptr()
        wt = _DTYPES.get(kind)
        if wt is None or kinds not in (None, kind) or w_post.shape != (H,) or not w_post.is_contiguous():
            return None
    kind, gt, gr = GATE_NONE, BF16, _NONE
    if gate is not None:
        gt, gs = _DTYPES.get(gate.dtype), gate.shape
        if gt is None or len(gs) != 2:
            return None
        kind = GATE_TOKEN if gs == (T, 1) else GATE_CHANNEL if gs == (1, H) else GATE_FULL
        if kind == GATE_FULL:
            gr = _rows(gate, shape, gate.dtype)
        else:
            gr = (gate.data_ptr(), 0) if gate.is_contiguous() else None
        if gr is None:
            return None
    return _NORM_ARGS.pack(_NORM_ARGS.size, xt, wt, gt, kind, 1 if gate_sigmoid else 0, residual_scale, weight_offset, eps,
                           T, H, *xr, *br, *gr, post, pre, *yr, *nr, status)


def moe_norm_forward(x, b, gate, w_post, w_pre, y, n, residual_scale: float = 1.0, weight_offset: float = 0.0,
                     eps: float = 1e-6, gate_sigmoid: bool = False, stream=None, check=True,
                     status: torch.Tensor = None) -> int:
    """y = residual_scale x + g norm(b; w_post), n = norm(y; w_pre); b, gate, w_post, w_pre, y and n may be None as
    include/moe_norm.h says.  gate [T, 1], [1, H] or [T, H]; x and y bf16 or float32, b and n bf16; status: 64 bytes for
    moe_get_device_status."""
    words = 0 if status is None else status.data_ptr()
    a = _norm_args(x, b, gate, w_post, w_pre, y, n, residual_scale, weight_offset, eps, gate_sigmoid, words)
    if a is None or (status is not None and (status.nbytes < 64 or not status.is_contiguous())):
        return _invalid("moe_norm_forward", check)
    rc = lib.moe_norm_forward(a, _stream(stream))
    if check:
        _check(rc, "moe_norm_forward")
    return rc


def _column_sum(t, H: int):
    """Pointer of a contiguous float32 [H] (0 for None); None if it is not one."""
    if t is None:
        return 0
    return t.data_ptr() if t.dtype is torch.float32 and t.shape == (H,) and t.is_contiguous() else None


def moe_norm_workspace_size(T: int, H: int) -> int:
    return int(lib.moe_norm_workspace_size(T, H))


def moe_norm_backward(y, b, gate, w_post, w_pre, dy, dn, workspace, dx=None, db=None, dgate=None, dw_post=None, dw_pre=None,
                      residual_scale: float = 1.0, weight_offset: float = 0.0, eps: float = 1e-6,
                      gate_sigmoid: bool = False, stream=None, check=True) -> int:
    """Gradients of moe_norm_forward from dy and dn; y is its y (without b: its x).  Outputs that are None are not
    computed; dgate has the gate's shape and type, dw_post and dw_pre are float32 [H]."""
    a = _norm_args(y, b, gate, w_post, w_pre, None, None, residual_scale, weight_offset, eps, gate_sigmoid)
    shape, dtype = y.shape, y.dtype
    dyr = _NONE if dy is None else _rows(dy, shape, dtype)
    dnr = _NONE if dn is None else _rows(dn, shape)
    dxr = _NONE if dx is None else _rows(dx, shape, dtype)
    dbr = _NONE if db is None else _rows(db, shape)
    if dgate is None:
        dgr = _NONE
    elif gate is None or dgate.dtype is not gate.dtype or dgate.shape != gate.shape:
        dgr = None
    elif dgate.shape == shape:
        dgr = _rows(dgate, shape, dgate.dtype)
    else:
        dgr = (dgate.data_ptr(), 0) if dgate.is_contiguous() else None
    post, pre = _column_sum(dw_post, shape[1]), _column_sum(dw_pre, shape[1])
    if None in (a, dyr, dnr, dxr, dbr, dgr, post, pre):
        return _invalid("moe_norm_backward", check)
    g = _NORM_GRADS.pack(_NORM_GRADS.size, *dyr, *dnr, *dxr, *dbr, *dgr, post, pre, workspace.data_ptr(), workspace.nbytes)
    rc = lib.moe_norm_backward(a, g, _stream(stream))
    if check:
        _check(rc, "moe_norm_backward")
    return rc


# ---------------------------------------------------------------- AdamW over many tensors (include/moe_adamw.h)

def moe_adamw_step(table: np.ndarray, p_dtype: int, g_dtype: int, state_bits: int, lr: float, beta1: float, beta2: float,
                   eps: float, weight_decay: float, step: int, grad_scale: torch.Tensor = None, stream=None,
                   check=True, address: int = None) -> int:
    """One step over the tensors of ``table`` (a contiguous array of ADAMW_TENSOR: sizes and device pointers); address:
    table.ctypes.data, for a caller that keeps it (asking NumPy takes 0.8 us)."""
    if table.dtype != ADAMW_TENSOR or not table.flags.c_contiguous or \
            (grad_scale is not None and (grad_scale.dtype != torch.float32 or grad_scale.numel() != 1)):
        return _invalid("moe_adamw_step", check)
    a = _ADAMW_ARGS.pack(_ADAMW_ARGS.size, table.size, address or table.ctypes.data, p_dtype, g_dtype, state_bits,
                         0 if grad_scale is None else grad_scale.data_ptr(), lr, beta1, beta2, eps, weight_decay, step)
    rc = lib.moe_adamw_step(a, _stream(stream))
    if check:
        _check(rc, "moe_adamw_step")
    return rc
