"""The gated feed-forward block (``include/gemm_ffn.h``):
``y = (act(x . w_gate^T) * (x . w_up^T)) . w_down^T`` and its gradients.

* ``gemm_ffn_forward(args)``, ``gemm_ffn_backward(args)``, ``gemm_ffn_plan(args, backward, num_cus)`` -- the C entry
  points on a ``GemmFfnArgs``.
* ``gated_ffn(x, w_gate, w_up, w_down)`` and ``gated_ffn_backward(dy, x, w_gate, w_up, w_down, gate, up)`` -- on torch
  tensors.

The torch-facing functions take workspaces, streams and results as the vocabulary
losses do (``loss.py``): the workspace from torch's allocator on the call's stream
unless given, nothing recorded for autograd.
"""
from __future__ import annotations

import ctypes
import functools

from . import _check, _lib, current_stream_word, layout_word
from .loss import _cus, _on, _rows, _warn_of_no_graph

try:
    import torch
except ImportError:   # the C entry points need no torch
    torch = None

GEMM_FFN_SILU = 0
GEMM_FFN_GELU = 1
GEMM_FFN_RELU = 2
GEMM_FFN_DW_SAME = 0
GEMM_FFN_DW_FP32 = 1
GEMM_FFN_DW_FP32_ADD = 2
GEMM_FFN_MAX_T = 1 << 24
GEMM_FFN_MAX_H = 1 << 20
GEMM_FFN_MAX_F = 1 << 20
GEMM_FFN_MAX_TH = 1 << 37

ACTIVATIONS = {"silu": GEMM_FFN_SILU, "gelu": GEMM_FFN_GELU, "relu": GEMM_FFN_RELU}


class GemmFfnArgs(ctypes.Structure):
    _fields_ = [
        ("x", ctypes.c_void_p), ("w_gate", ctypes.c_void_p), ("w_up", ctypes.c_void_p), ("w_down", ctypes.c_void_p),
        ("T", ctypes.c_int64), ("H", ctypes.c_int64), ("F", ctypes.c_int64),
        ("ldx", ctypes.c_int64), ("ldw_gate", ctypes.c_int64), ("ldw_up", ctypes.c_int64), ("ldw_down", ctypes.c_int64),
        ("layout", ctypes.c_uint32), ("act", ctypes.c_uint32),
        ("gate", ctypes.c_void_p), ("up", ctypes.c_void_p), ("ldgate", ctypes.c_int64), ("ldup", ctypes.c_int64),
        ("y", ctypes.c_void_p), ("ldy", ctypes.c_int64),
        ("dy", ctypes.c_void_p), ("lddy", ctypes.c_int64),
        ("dx", ctypes.c_void_p), ("lddx", ctypes.c_int64),
        ("dw_gate", ctypes.c_void_p), ("dw_up", ctypes.c_void_p), ("dw_down", ctypes.c_void_p),
        ("lddw_gate", ctypes.c_int64), ("lddw_up", ctypes.c_int64), ("lddw_down", ctypes.c_int64),
        ("dw_type", ctypes.c_uint32), ("num_cus", ctypes.c_int32),
        ("stream", ctypes.c_void_p), ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t),
    ]


class GemmFfnPlan(ctypes.Structure):
    _fields_ = [
        ("num_cus", ctypes.c_int32), ("parts", ctypes.c_int32),
        ("first_tile_f", ctypes.c_int32), ("first_tile_t", ctypes.c_int32),
        ("out_tile_h", ctypes.c_int32), ("out_tile_t", ctypes.c_int32), ("out_splits", ctypes.c_int32),
        ("dw_tile_p", ctypes.c_int32), ("dw_tile_q", ctypes.c_int32), ("dw_splits", ctypes.c_int32),
        ("workspace_bytes", ctypes.c_int64),
    ]


_lib.gemm_ffn_plan.restype = ctypes.c_int
_lib.gemm_ffn_plan.argtypes = [ctypes.POINTER(GemmFfnArgs), ctypes.c_int32, ctypes.c_int32, ctypes.POINTER(GemmFfnPlan)]
_lib.gemm_ffn_forward.restype = ctypes.c_int
_lib.gemm_ffn_forward.argtypes = [ctypes.POINTER(GemmFfnArgs)]
_lib.gemm_ffn_backward.restype = ctypes.c_int
_lib.gemm_ffn_backward.argtypes = [ctypes.POINTER(GemmFfnArgs)]


# ---- C entry points, same names ----------------------------------------------------
def gemm_ffn_forward(args: GemmFfnArgs) -> int:
    """Raw call; returns the status (no exception)."""
    return _lib.gemm_ffn_forward(ctypes.byref(args))


def gemm_ffn_backward(args: GemmFfnArgs) -> int:
    return _lib.gemm_ffn_backward(ctypes.byref(args))


def gemm_ffn_plan(args: GemmFfnArgs, backward: bool, num_cus: int) -> GemmFfnPlan:
    p = GemmFfnPlan()
    _check(_lib.gemm_ffn_plan(ctypes.byref(args), int(backward), num_cus, ctypes.byref(p)))
    return p


# ---- on torch tensors ------------------------------------------------------------------
def _block(x, w_gate, w_up, w_down, activation, b_layout):
    """GemmFfnArgs with the block's inputs filled in."""
    if any(t.dim() != 2 for t in (x, w_gate, w_up, w_down)):
        raise ValueError("x and the weights must be 2-D")
    if x.dtype not in (torch.bfloat16, torch.float16):
        raise TypeError("x must be bf16 or fp16")
    if not x.is_cuda:
        raise ValueError("x must be a device tensor")
    if b_layout not in ("nk", "kn"):
        raise ValueError("b_layout must be 'kn' or 'nk'")
    if activation not in ACTIVATIONS:
        raise ValueError(f"activation must be one of {sorted(ACTIVATIONS)}")
    a = GemmFfnArgs()
    a.T, a.H = x.shape
    a.F = w_gate.shape[0] if b_layout == "nk" else w_gate.shape[1]
    a.layout = layout_word(b_layout, "bf16" if x.dtype == torch.bfloat16 else "fp16")
    a.act = ACTIVATIONS[activation]
    a.x, a.ldx = x.data_ptr(), _rows("x", x, a.T, a.H, x.dtype, x.device)
    inner, outer = ((a.F, a.H), (a.H, a.F)) if b_layout == "nk" else ((a.H, a.F), (a.F, a.H))
    a.w_gate, a.ldw_gate = w_gate.data_ptr(), _rows("w_gate", w_gate, *inner, x.dtype, x.device)
    a.w_up, a.ldw_up = w_up.data_ptr(), _rows("w_up", w_up, *inner, x.dtype, x.device)
    a.w_down, a.ldw_down = w_down.data_ptr(), _rows("w_down", w_down, *outer, x.dtype, x.device)
    return a


def _hidden(a, x, gate, up):
    a.gate, a.ldgate = gate.data_ptr(), _rows("gate", gate, a.T, a.F, x.dtype, x.device)
    a.up, a.ldup = up.data_ptr(), _rows("up", up, a.T, a.F, x.dtype, x.device)


@functools.lru_cache(maxsize=1024)
def _workspace_bytes(T, H, F, layout, ldw_gate, ldw_up, dx, dw_gate, dw_up, dw_down, dw_type, backward, cus):
    a = GemmFfnArgs(T=T, H=H, F=F, layout=layout, ldw_gate=ldw_gate, ldw_up=ldw_up, dx=dx, dw_gate=dw_gate, dw_up=dw_up, dw_down=dw_down, dw_type=dw_type)
    return gemm_ffn_plan(a, backward, cus).workspace_bytes


def _call(a, x, backward, workspace):
    """Runs the call on torch's current stream, its workspace torch's unless given."""
    device = x.device
    a.stream = current_stream_word(device.index)
    if workspace is None:
        a.num_cus = cus = _cus(device.index)
        need = _workspace_bytes(a.T, a.H, a.F, a.layout, a.ldw_gate, a.ldw_up, 1 if a.dx else 0, 1 if a.dw_gate else 0,
                                1 if a.dw_up else 0, 1 if a.dw_down else 0, a.dw_type, backward, cus)
        workspace = torch.empty(need or 1, dtype=torch.uint8, device=device)
        a.workspace_bytes = need
    elif not workspace.is_cuda or workspace.device != device or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on x's device")
    else:
        a.workspace_bytes = workspace.numel() * workspace.element_size()
    a.workspace = workspace.data_ptr()
    _check((_lib.gemm_ffn_backward if backward else _lib.gemm_ffn_forward)(ctypes.byref(a)))


def gated_ffn(x, w_gate, w_up, w_down, *, activation: str = "silu", b_layout: str = "nk", save: bool = False, y=None,
              gate=None, up=None, workspace=None, stream=None):
    """``y = (act(x . w_gate^T) * (x . w_up^T)) . w_down^T``, [T,H] of x's dtype.

    x [T,H]; "nk": w_gate, w_up [F,H] and w_down [H,F]; "kn": each transposed.
    All bf16 or all fp16 on one device, rows contiguous at any stride that is a
    multiple of 8 elements; H and F multiples of 8.  activation: "silu", "gelu"
    (the exact form) or "relu".  ``save`` (or ``gate`` and ``up`` given): returns
    ``(y, gate, up)``, the two first products [T,F] that the backward call needs,
    else ``y``.  Nothing is recorded for autograd.  Enqueues on ``stream`` or
    torch's current stream.
    """
    _warn_of_no_graph(x, w_gate, w_up, w_down, what="the block")
    a = _block(x, w_gate, w_up, w_down, activation, b_layout)
    if (gate is None) != (up is None):
        raise ValueError("gate and up are given both or neither")
    save = save or gate is not None
    with _on(x, stream):
        y = x.new_empty((a.T, a.H)) if y is None else y
        a.y, a.ldy = y.data_ptr(), _rows("y", y, a.T, a.H, x.dtype, x.device)
        if save:
            if gate is None:
                gate = x.new_empty((a.T, a.F))
                up = torch.empty_like(gate)
            _hidden(a, x, gate, up)
        _call(a, x, False, workspace)
    return (y, gate, up) if save else y


def gated_ffn_backward(dy, x, w_gate, w_up, w_down, gate, up, *, activation: str = "silu", b_layout: str = "nk",
                       dx=None, dw_gate=None, dw_up=None, dw_down=None, need_dx: bool = True, need_dw: bool = True,
                       accumulate_dw: bool = False, workspace=None, stream=None):
    """``(dx, dw_gate, dw_up, dw_down)`` of ``gated_ffn`` for the gradient ``dy`` [T,H] of its result.

    ``gate`` and ``up`` are what the forward call kept.  dx [T,H] has x's dtype;
    the weights' gradients have the weights' shapes and dtype, or are given fp32
    tensors, all three of one dtype (``accumulate_dw``: added to).  ``need_dx`` /
    ``need_dw`` false: not computed (None).
    """
    a = _block(x, w_gate, w_up, w_down, activation, b_layout)
    a.dy, a.lddy = dy.data_ptr(), _rows("dy", dy, a.T, a.H, x.dtype, x.device)
    _hidden(a, x, gate, up)
    given = [t for t in (dw_gate, dw_up, dw_down) if t is not None]
    if not need_dx and dx is not None or not need_dw and given:
        raise ValueError("dx or weights' gradients given but not needed")
    if given and (len(given) < 3 or len({t.dtype for t in given}) > 1):
        raise ValueError("the weights' gradients are given all or none, of one dtype")
    if accumulate_dw and (not given or dw_gate.dtype != torch.float32):
        raise ValueError("accumulate_dw needs fp32 gradients to add to")
    with _on(x, stream):
        if need_dx:
            dx = torch.empty_like(x) if dx is None else dx
            a.dx, a.lddx = dx.data_ptr(), _rows("dx", dx, a.T, a.H, x.dtype, x.device)
        if need_dw:
            if not given:
                dw_gate, dw_up, dw_down = torch.empty_like(w_gate), torch.empty_like(w_up), torch.empty_like(w_down)
            fp32 = dw_gate.dtype == torch.float32
            dtype = torch.float32 if fp32 else x.dtype
            a.dw_gate, a.lddw_gate = dw_gate.data_ptr(), _rows("dw_gate", dw_gate, *w_gate.shape, dtype, x.device)
            a.dw_up, a.lddw_up = dw_up.data_ptr(), _rows("dw_up", dw_up, *w_up.shape, dtype, x.device)
            a.dw_down, a.lddw_down = dw_down.data_ptr(), _rows("dw_down", dw_down, *w_down.shape, dtype, x.device)
            if fp32:
                a.dw_type = GEMM_FFN_DW_FP32_ADD if accumulate_dw else GEMM_FFN_DW_FP32
        _call(a, x, True, workspace)
    return dx, dw_gate, dw_up, dw_down
