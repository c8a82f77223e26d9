"""A shared projection with a low-rank adapter per row (``include/gemm_lora.h``):
``y_t = x_t . w^T + scale[a_t] (x_t . a[a_t]^T) . b[a_t]^T`` and its gradients.

* ``gemm_lora_forward(args)``, ``gemm_lora_backward(args)``, ``gemm_lora_plan(args, backward, num_cus)`` -- the C entry
  points on a ``GemmLoraArgs``.
* ``linear_lora(x, w, a, b, adapter)`` and ``linear_lora_backward(dy, x, w, a, b, adapter)`` -- on torch tensors.

The torch-facing functions take workspaces, streams and results as the vocabulary
losses do (``loss.py``): the workspace from torch's allocator on the call's stream
unless given, nothing recorded for autograd.
"""
from __future__ import annotations

import ctypes
import functools

from . import _check, _lib, current_stream_word, layout_word
from .loss import _cus, _on, _rows, _vector, _warn_of_no_graph

try:
    import torch
except ImportError:   # the C entry points need no torch
    torch = None

GEMM_LORA_DAB_SAME = 0
GEMM_LORA_DAB_FP32 = 1
GEMM_LORA_DAB_FP32_ADD = 2
GEMM_LORA_MAX_T = 1 << 24
GEMM_LORA_MAX_H = 1 << 20
GEMM_LORA_MAX_R = 1024
GEMM_LORA_MAX_ADAPTERS = 1 << 16
GEMM_LORA_MAX_TH = 1 << 37
GEMM_LORA_MAX_LT = 1 << 34
GEMM_LORA_MAX_LRH = 1 << 38
GEMM_LORA_MAX_TR = 1 << 31
GEMM_LORA_MAX_TILES = 1 << 23
GEMM_LORA_MAX_STRIDE = 1 << 40


class GemmLoraArgs(ctypes.Structure):
    _fields_ = [
        ("x", ctypes.c_void_p), ("w", ctypes.c_void_p), ("a", ctypes.c_void_p), ("b", ctypes.c_void_p),
        ("adapter", ctypes.c_void_p), ("scale", ctypes.c_void_p),
        ("T", ctypes.c_int64), ("H", ctypes.c_int64), ("N", ctypes.c_int64),
        ("R", ctypes.c_int32), ("adapters", ctypes.c_int32),
        ("ldx", ctypes.c_int64), ("ldw", ctypes.c_int64), ("stride_a", ctypes.c_int64), ("stride_b", ctypes.c_int64),
        ("layout", ctypes.c_uint32), ("dab_type", ctypes.c_uint32),
        ("y", ctypes.c_void_p), ("ldy", ctypes.c_int64),
        ("dy", ctypes.c_void_p), ("lddy", ctypes.c_int64),
        ("dx", ctypes.c_void_p), ("lddx", ctypes.c_int64),
        ("da", ctypes.c_void_p), ("db", ctypes.c_void_p),
        ("num_cus", ctypes.c_int32),
        ("stream", ctypes.c_void_p), ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t),
    ]


class GemmLoraPlan(ctypes.Structure):
    _fields_ = [
        ("num_cus", ctypes.c_int32),
        ("low_tile_r", ctypes.c_int32), ("low_splits", ctypes.c_int32), ("low_lists", ctypes.c_int32),
        ("out_tile_p", ctypes.c_int32), ("out_tile_t", ctypes.c_int32), ("out_splits", ctypes.c_int32),
        ("dab_splits", ctypes.c_int32), ("out_whole", ctypes.c_int64), ("workspace_bytes", ctypes.c_int64),
    ]


_lib.gemm_lora_plan.restype = ctypes.c_int
_lib.gemm_lora_plan.argtypes = [ctypes.POINTER(GemmLoraArgs), ctypes.c_int32, ctypes.c_int32, ctypes.POINTER(GemmLoraPlan)]
_lib.gemm_lora_forward.restype = ctypes.c_int
_lib.gemm_lora_forward.argtypes = [ctypes.POINTER(GemmLoraArgs)]
_lib.gemm_lora_backward.restype = ctypes.c_int
_lib.gemm_lora_backward.argtypes = [ctypes.POINTER(GemmLoraArgs)]


# ---- C entry points, same names ----------------------------------------------------
def gemm_lora_forward(args: GemmLoraArgs) -> int:
    """Raw call; returns the status (no exception)."""
    return _lib.gemm_lora_forward(ctypes.byref(args))


def gemm_lora_backward(args: GemmLoraArgs) -> int:
    return _lib.gemm_lora_backward(ctypes.byref(args))


def gemm_lora_plan(args: GemmLoraArgs, backward: bool, num_cus: int) -> GemmLoraPlan:
    p = GemmLoraPlan()
    _check(_lib.gemm_lora_plan(ctypes.byref(args), int(backward), num_cus, ctypes.byref(p)))
    return p


# ---- on torch tensors ------------------------------------------------------------------
def _matrices(name, t, count, rows, cols, dtype, device):
    """The element stride between the packed matrices of a [count, rows, cols] tensor."""
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}")
    if t.shape != (count, rows, cols):
        raise ValueError(f"{name} must be [{count}, {rows}, {cols}]")
    if t.is_contiguous():
        return 0
    stride = t.stride()
    if cols > 1 and stride[2] != 1 or rows > 1 and stride[1] != cols:
        raise ValueError(f"{name}: every adapter's matrix must be contiguous")
    if count <= 1:
        return 0
    if stride[0] < rows * cols:   # an expanded tensor; 0 would mean packed
        raise ValueError(f"{name}: adapters overlap")
    return stride[0]


def _projection(x, w, a, b, adapter, scale, b_layout):
    """GemmLoraArgs with the projection's inputs filled in."""
    if x.dim() != 2 or w.dim() != 2 or a.dim() != 3 or b.dim() != 3:
        raise ValueError("x and w must be 2-D, a and b 3-D")
    if x.dtype not in (torch.bfloat16, torch.float16):
        raise TypeError("x must be bf16 or fp16")
    if not x.is_cuda:
        raise ValueError("x must be a device tensor")
    if b_layout not in ("nk", "kn"):
        raise ValueError("b_layout must be 'kn' or 'nk'")
    nk = b_layout == "nk"
    p = GemmLoraArgs()
    p.T, p.H = x.shape
    p.N = w.shape[0] if nk else w.shape[1]
    p.adapters = a.shape[0]
    p.R = a.shape[1] if nk else a.shape[2]
    p.layout = layout_word(b_layout, "bf16" if x.dtype == torch.bfloat16 else "fp16")
    p.x, p.ldx = x.data_ptr(), _rows("x", x, p.T, p.H, x.dtype, x.device)
    p.w, p.ldw = w.data_ptr(), _rows("w", w, *((p.N, p.H) if nk else (p.H, p.N)), x.dtype, x.device)
    p.a, p.stride_a = a.data_ptr(), _matrices("a", a, p.adapters, *((p.R, p.H) if nk else (p.H, p.R)), x.dtype, x.device)
    p.b, p.stride_b = b.data_ptr(), _matrices("b", b, p.adapters, *((p.N, p.R) if nk else (p.R, p.N)), x.dtype, x.device)
    p.adapter = _vector("adapter", adapter, (p.T,), torch.int64, x.device)
    if scale is not None:
        p.scale = _vector("scale", scale, (p.adapters,), torch.float32, x.device)
    return p


@functools.lru_cache(maxsize=1024)
def _workspace_bytes(T, H, N, R, adapters, layout, dx, da, db, dab_type, backward, cus):
    p = GemmLoraArgs(T=T, H=H, N=N, R=R, adapters=adapters, layout=layout, dx=dx, da=da, db=db, dab_type=dab_type)
    return gemm_lora_plan(p, backward, cus).workspace_bytes


def _call(p, x, backward, workspace):
    """Runs the call on torch's current stream, its workspace torch's unless given."""
    device = x.device
    p.stream = current_stream_word(device.index)
    if workspace is None:
        p.num_cus = cus = _cus(device.index)
        need = _workspace_bytes(p.T, p.H, p.N, p.R, p.adapters, p.layout, 1 if p.dx else 0, 1 if p.da else 0, 1 if p.db else 0,
                                p.dab_type, backward, cus)
        workspace = torch.empty(need or 1, dtype=torch.uint8, device=device)
        p.workspace_bytes = need
    elif not workspace.is_cuda or workspace.device != device or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on x's device")
    else:
        p.workspace_bytes = workspace.numel() * workspace.element_size()
    p.workspace = workspace.data_ptr()
    _check((_lib.gemm_lora_backward if backward else _lib.gemm_lora_forward)(ctypes.byref(p)))


def linear_lora(x, w, a, b, adapter, *, scale=None, b_layout: str = "nk", y=None, workspace=None, stream=None):
    """``x . w^T`` with each row's adapter added, [T,N] of x's dtype.

    x [T,H]; "nk": w [N,H], a [L,R,H] and b [L,N,R]; "kn": each matrix
    transposed.  All bf16 or all fp16 on one device; rows of x and w contiguous
    at any stride that is a multiple of 8 elements, adapters packed; H, N and R
    multiples of 8.  adapter: int64 [T], negative: none; rows of one request lie
    best together.  scale: fp32 [L].  A row whose adapter is L or more is NaN.
    What an adapter holds, an infinity or NaN too, reaches the rows that name it alone.
    Nothing is recorded for autograd.  Enqueues on ``stream`` or torch's current
    stream.
    """
    _warn_of_no_graph(x, w, a, b, what="the projection")
    p = _projection(x, w, a, b, adapter, scale, b_layout)
    with _on(x, stream):
        y = x.new_empty((p.T, p.N)) if y is None else y
        p.y, p.ldy = y.data_ptr(), _rows("y", y, p.T, p.N, x.dtype, x.device)
        _call(p, x, False, workspace)
    return y


def linear_lora_backward(dy, x, w, a, b, adapter, *, scale=None, b_layout: str = "nk", dx=None, da=None, db=None,
                         need_dx: bool = True, need_dab: bool = True, accumulate_dab: bool = False, workspace=None,
                         stream=None):
    """``(dx, da, db)`` of ``linear_lora`` for the gradient ``dy`` [T,N] of its result.

    dx [T,H] has x's dtype; da and db have a's and b's shapes and dtype, or are
    given fp32 tensors (``accumulate_dab``: added to); adapters that no row names
    get zeros.  w is shared and has no gradient here.  ``need_dx`` / ``need_dab``
    false: not computed (None).
    """
    p = _projection(x, w, a, b, adapter, scale, b_layout)
    p.dy, p.lddy = dy.data_ptr(), _rows("dy", dy, p.T, p.N, x.dtype, x.device)
    if not need_dx and dx is not None or not need_dab and (da is not None or db is not None):
        raise ValueError("dx, da or db given but not needed")
    if (da is None) != (db is None) or da is not None and da.dtype != db.dtype:
        raise ValueError("da and db are given both or neither, of one dtype")
    if accumulate_dab and (da is None or da.dtype != torch.float32):
        raise ValueError("accumulate_dab needs fp32 gradients to add to")
    with _on(x, stream):
        if need_dx:
            dx = torch.empty_like(x) if dx is None else dx
            p.dx, p.lddx = dx.data_ptr(), _rows("dx", dx, p.T, p.H, x.dtype, x.device)
        if need_dab:
            if da is None:
                da, db = a.new_empty(a.shape), b.new_empty(b.shape)   # packed, as a and b need not be
            dtype = torch.float32 if da.dtype == torch.float32 else x.dtype
            p.da, p.db = _vector("da", da, a.shape, dtype, x.device), _vector("db", db, b.shape, dtype, x.device)
            if dtype == torch.float32:
                p.dab_type = GEMM_LORA_DAB_FP32_ADD if accumulate_dab else GEMM_LORA_DAB_FP32
        _call(p, x, True, workspace)
    return dx, da, db
