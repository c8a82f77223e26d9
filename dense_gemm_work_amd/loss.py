"""Vocabulary losses (``include/gemm_loss.h``): softmax cross entropy and top-k
distillation over the logits ``x . w^T``, which are never kept.

* ``gemm_loss_forward(args)``, ``gemm_loss_backward(args)``, ``gemm_loss_plan(args, backward, num_cus)`` -- the C
  entry points on a ``GemmLossArgs``.
* ``linear_cross_entropy(x, w, target)`` and ``linear_cross_entropy_backward(grad, x, w, target, lse)``,
  ``linear_distill(x, w, teacher_index, teacher_logits)`` and ``linear_distill_backward(...)`` -- on torch tensors.

The torch-facing functions take their workspace from torch's allocator on the
call's stream (so calls on different streams, and graphs captured separately, do
not share one), unless ``workspace`` is given.  They record nothing for autograd:
the backward calls are the gradients, and a forward call whose inputs require
gradients while they are being recorded warns that its loss has none.  With ``stream`` given, the inputs must be
ready on it and stay allocated until it has run the call (``record_stream`` on
them says so to torch's allocator); results not given are allocated on it.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import warnings

from . import _check, _lib, layout_word, stream_word

try:
    import torch
    from torch.autograd import forward_ad
except ImportError:   # the C entry points need no torch
    torch = None

GEMM_LOSS_XENT = 0
GEMM_LOSS_DISTILL = 1
GEMM_LOSS_FP32 = 0
GEMM_LOSS_BF16 = 1
GEMM_LOSS_FP16 = 2
GEMM_LOSS_DW_SAME = 0
GEMM_LOSS_DW_FP32 = 1
GEMM_LOSS_DW_FP32_ADD = 2
GEMM_LOSS_MAX_T = 1 << 24
GEMM_LOSS_MAX_V = 1 << 21
GEMM_LOSS_MAX_H = 1 << 20
GEMM_LOSS_MAX_ENTRIES = 1024
GEMM_LOSS_MAX_TV = 1 << 37
GEMM_LOSS_MAX_TH = 1 << 37


class GemmLossArgs(ctypes.Structure):
    _fields_ = [
        ("x", ctypes.c_void_p), ("w", ctypes.c_void_p),
        ("T", ctypes.c_int64), ("V", ctypes.c_int64), ("H", ctypes.c_int64),
        ("ldx", ctypes.c_int64), ("ldw", ctypes.c_int64),
        ("layout", ctypes.c_uint32), ("kind", ctypes.c_uint32),
        ("target", ctypes.c_void_p), ("ignore_index", ctypes.c_int64),
        ("z_loss", ctypes.c_float), ("entries", ctypes.c_int32),
        ("teacher_index", ctypes.c_void_p), ("teacher_logits", ctypes.c_void_p),
        ("teacher_type", ctypes.c_uint32), ("temperature", ctypes.c_float),
        ("loss", ctypes.c_void_p), ("lse", ctypes.c_void_p), ("grad", ctypes.c_void_p),
        ("dx", ctypes.c_void_p), ("lddx", ctypes.c_int64),
        ("dw", ctypes.c_void_p), ("lddw", ctypes.c_int64),
        ("dw_type", ctypes.c_uint32), ("num_cus", ctypes.c_int32),
        ("stream", ctypes.c_void_p), ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t),
    ]


class GemmLossPlan(ctypes.Structure):
    _fields_ = [
        ("tile_v", ctypes.c_int32), ("tile_t", ctypes.c_int32), ("num_cus", ctypes.c_int32),
        ("pieces", ctypes.c_int32), ("piece", ctypes.c_int64),
        ("dx_tile_h", ctypes.c_int32), ("dx_tile_t", ctypes.c_int32), ("dx_splits", ctypes.c_int32),
        ("dw_tile_p", ctypes.c_int32), ("dw_tile_q", ctypes.c_int32), ("dw_splits", ctypes.c_int32),
        ("workspace_bytes", ctypes.c_int64),
    ]


_lib.gemm_loss_plan.restype = ctypes.c_int
_lib.gemm_loss_plan.argtypes = [ctypes.POINTER(GemmLossArgs), ctypes.c_int32, ctypes.c_int32,
                                ctypes.POINTER(GemmLossPlan)]
_lib.gemm_loss_forward.restype = ctypes.c_int
_lib.gemm_loss_forward.argtypes = [ctypes.POINTER(GemmLossArgs)]
_lib.gemm_loss_backward.restype = ctypes.c_int
_lib.gemm_loss_backward.argtypes = [ctypes.POINTER(GemmLossArgs)]


# ---- C entry points, same names ----------------------------------------------------
def gemm_loss_forward(args: GemmLossArgs) -> int:
    """Raw call; returns the status (no exception)."""
    return _lib.gemm_loss_forward(ctypes.byref(args))


def gemm_loss_backward(args: GemmLossArgs) -> int:
    return _lib.gemm_loss_backward(ctypes.byref(args))


def gemm_loss_plan(args: GemmLossArgs, backward: bool, num_cus: int) -> GemmLossPlan:
    p = GemmLossPlan()
    _check(_lib.gemm_loss_plan(ctypes.byref(args), int(backward), num_cus, ctypes.byref(p)))
    return p


_NOTHING = contextlib.nullcontext()


# ---- on torch tensors ------------------------------------------------------------------
def _rows(name, t, rows, cols, dtype, device):
    """The element stride between the rows of a [rows, cols] tensor whose rows are contiguous."""
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}")
    if t.shape != (rows, cols):
        raise ValueError(f"{name} must be [{rows}, {cols}]")
    step, unit = t.stride()
    if unit != 1 and cols > 1 and rows > 0:
        raise ValueError(f"{name}: every row must be contiguous")
    if rows <= 1:
        return 0
    if step < cols:   # an expanded tensor; 0 would mean packed
        raise ValueError(f"{name}: rows overlap")
    return step


def _vector(name, t, shape, dtypes, device):
    if t.dtype not in (dtypes if isinstance(dtypes, tuple) else (dtypes,)):
        raise TypeError(f"{name} must be {dtypes}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}")
    if t.shape != tuple(shape) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {list(shape)}")
    return t.data_ptr()


def _product(x, w, b_layout):
    """GemmLossArgs with the product's part filled in."""
    if x.dim() != 2 or w.dim() != 2:
        raise ValueError("x and w must be 2-D")
    if x.dtype not in (torch.bfloat16, torch.float16) or w.dtype != x.dtype:
        raise TypeError("x and w must both be bf16 or both fp16")
    if not x.is_cuda:
        raise ValueError("x must be a device tensor")
    if b_layout not in ("nk", "kn"):
        raise ValueError("b_layout must be 'kn' or 'nk'")
    a = GemmLossArgs()
    a.T, a.H = x.shape
    a.V = w.shape[0] if b_layout == "nk" else w.shape[1]
    a.layout = layout_word(b_layout, "bf16" if x.dtype == torch.bfloat16 else "fp16")
    a.x, a.ldx = x.data_ptr(), _rows("x", x, a.T, a.H, x.dtype, x.device)
    a.w, a.ldw = w.data_ptr(), _rows("w", w, *((a.V, a.H) if b_layout == "nk" else (a.H, a.V)), x.dtype, x.device)
    return a


def _warn_of_no_graph(*inputs, what="the loss"):
    if torch.is_grad_enabled() and any(t.requires_grad for t in inputs):
        warnings.warn(f"{what} is not recorded for autograd: its gradients come from the _backward call "
                      "(pass detached tensors, or call under torch.no_grad())", stacklevel=3)
    if forward_ad._current_level >= 0 and any(forward_ad.unpack_dual(t).tangent is not None for t in inputs):
        warnings.warn(f"{what} has no forward-mode derivative: the tangents of its inputs are dropped", stacklevel=3)


def _xent(a, x, target, ignore_index, z_loss):
    a.kind = GEMM_LOSS_XENT
    a.target = _vector("target", target, (a.T,), torch.int64, x.device)
    a.ignore_index = ignore_index
    a.z_loss = z_loss


def _distill(a, x, teacher_index, teacher_logits, temperature):
    types = {torch.float32: GEMM_LOSS_FP32, torch.bfloat16: GEMM_LOSS_BF16, torch.float16: GEMM_LOSS_FP16}
    if teacher_index.dim() != 2:
        raise ValueError("teacher_index must be [T, K]")
    a.kind = GEMM_LOSS_DISTILL
    a.entries = teacher_index.shape[1]
    a.teacher_index = _vector("teacher_index", teacher_index, (a.T, a.entries), torch.int64, x.device)
    a.teacher_logits = _vector("teacher_logits", teacher_logits, (a.T, a.entries), tuple(types), x.device)
    a.teacher_type = types[teacher_logits.dtype]
    a.temperature = temperature


@functools.lru_cache(maxsize=None)
def _cus(index):
    return torch.cuda.get_device_properties(index).multi_processor_count


@functools.lru_cache(maxsize=1024)
def _workspace_bytes(T, V, H, layout, kind, entries, dx, dw, dw_type, backward, cus):
    a = GemmLossArgs(T=T, V=V, H=H, layout=layout, kind=kind, entries=entries, dx=dx, dw=dw, dw_type=dw_type)
    return gemm_loss_plan(a, backward, cus).workspace_bytes


def _call(a, x, backward, workspace, outputs):
    """Runs the call on torch's current stream, its workspace torch's unless given."""
    device = x.device
    a.stream = stream_word(torch.cuda.current_stream(device))
    if workspace is None:
        a.num_cus = cus = _cus(device.index)
        need = _workspace_bytes(a.T, a.V, a.H, a.layout, a.kind, a.entries, 1 if a.dx else 0, 1 if a.dw else 0,
                                a.dw_type, backward, cus)
        workspace = torch.empty(need or 1, dtype=torch.uint8, device=device)
        a.workspace_bytes = need
    elif not workspace.is_cuda or workspace.device != device or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on x's device")
    else:
        a.workspace_bytes = workspace.numel() * workspace.element_size()
    a.workspace = workspace.data_ptr()
    _check((_lib.gemm_loss_backward if backward else _lib.gemm_loss_forward)(ctypes.byref(a)))
    return outputs


def _on(x, stream):
    """x's device and the call's stream made current."""
    if stream is not None:
        if stream.device != x.device:
            raise ValueError("stream must be on x's device")
        stack = contextlib.ExitStack()
        stack.enter_context(torch.cuda.device(x.device))
        stack.enter_context(torch.cuda.stream(stream))
        return stack
    if x.device.index == torch.cuda.current_device():
        return _NOTHING
    return torch.cuda.device(x.device)


def _forward(a, x, loss, lse, workspace, stream):
    with _on(x, stream):
        loss = torch.empty(a.T, dtype=torch.float32, device=x.device) if loss is None else loss
        lse = torch.empty(a.T, dtype=torch.float32, device=x.device) if lse is None else lse
        a.loss = _vector("loss", loss, (a.T,), torch.float32, x.device)
        a.lse = _vector("lse", lse, (a.T,), torch.float32, x.device)
        return _call(a, x, False, workspace, (loss, lse))


def _backward(a, x, w, grad, lse, dx, dw, need_dx, need_dw, accumulate_dw, workspace, stream):
    a.grad = _vector("grad", grad, (a.T,), torch.float32, x.device)
    a.lse = _vector("lse", lse, (a.T,), torch.float32, x.device)
    if not need_dx and dx is not None or not need_dw and dw is not None:
        raise ValueError("dx or dw given but not needed")
    if accumulate_dw and (dw is None or dw.dtype != torch.float32):
        raise ValueError("accumulate_dw needs an fp32 dw to add to")
    with _on(x, stream):
        if need_dx:
            dx = torch.empty((a.T, a.H), dtype=x.dtype, device=x.device) if dx is None else dx
            a.dx, a.lddx = dx.data_ptr(), _rows("dx", dx, a.T, a.H, x.dtype, x.device)
        if need_dw:
            dw = torch.empty(tuple(w.shape), dtype=w.dtype, device=x.device) if dw is None else dw
            fp32 = dw.dtype == torch.float32
            a.dw, a.lddw = dw.data_ptr(), _rows("dw", dw, *w.shape, torch.float32 if fp32 else x.dtype, x.device)
            if fp32:
                a.dw_type = GEMM_LOSS_DW_FP32_ADD if accumulate_dw else GEMM_LOSS_DW_FP32
        return _call(a, x, True, workspace, (dx, dw))


def linear_cross_entropy(x, w, target, *, b_layout: str = "nk", ignore_index: int = -100, z_loss: float = 0.0,
                         loss=None, lse=None, workspace=None, stream=None):
    """Per-row softmax cross entropy of the logits ``x . w^T`` (w [V,H], "nk") or ``x . w`` (w [H,V], "kn").

    ``loss[t] = lse[t] - logits[t, target[t]] + z_loss lse[t]^2``; rows whose
    target is ``ignore_index`` have loss 0.  Returns ``(loss, lse)``, fp32 [T];
    ``lse`` is what the backward call needs (neither is recorded for autograd).  A mean over the rows is
    ``loss.sum() / (target != ignore_index).sum()``, its backward call's ``grad``
    that divisor's inverse in every row.
    x [T,H], w: bf16 or fp16 on one device, rows contiguous at any stride that
    is a multiple of 8 elements; target: int64 [T].  A target out of range makes
    its row's loss NaN.  Rows that are left out may hold anything finite: their
    gradient is zero, and zero times infinity would be NaN in dw.  Enqueues on ``stream`` or torch's current stream;
    ``loss`` and ``lse`` may be given.
    """
    _warn_of_no_graph(x, w)
    a = _product(x, w, b_layout)
    _xent(a, x, target, ignore_index, z_loss)
    return _forward(a, x, loss, lse, workspace, stream)


def linear_cross_entropy_backward(grad, x, w, target, lse, *, b_layout: str = "nk", ignore_index: int = -100,
                                  z_loss: float = 0.0, dx=None, dw=None, need_dx: bool = True, need_dw: bool = True,
                                  accumulate_dw: bool = False, workspace=None, stream=None):
    """``(dx, dw)`` of ``linear_cross_entropy`` for the gradient ``grad`` (fp32 [T]) of each row's loss.

    dx [T,H] has x's dtype; dw has w's shape and dtype, or is a given fp32 tensor
    (``accumulate_dw``: added to).  ``need_dx`` / ``need_dw`` false: not computed
    (None).  ``lse`` is the forward call's.
    """
    a = _product(x, w, b_layout)
    _xent(a, x, target, ignore_index, z_loss)
    return _backward(a, x, w, grad, lse, dx, dw, need_dx, need_dw, accumulate_dw, workspace, stream)


def linear_distill(x, w, teacher_index, teacher_logits, *, temperature: float = 1.0, b_layout: str = "nk",
                   loss=None, lse=None, workspace=None, stream=None):
    """Per-row divergence of the logits ``x . w^T`` from a teacher's top logits.

    teacher_index: int64 [T,K] vocabulary entries (negative: padding);
    teacher_logits: [T,K], fp32, bf16 or fp16.  With
    ``q = softmax(teacher_logits / temperature)`` over a row's entries,
    ``loss[t] = temperature^2 sum_k q_k (log q_k - logits[t, index_k] / temperature + lse[t])``
    and ``lse[t] = logsumexp(logits[t] / temperature)``.  Rows without entries
    have loss 0.  Returns ``(loss, lse)``, fp32 [T].  x, w and the rest as for
    ``linear_cross_entropy``.
    """
    _warn_of_no_graph(x, w, teacher_logits)
    a = _product(x, w, b_layout)
    _distill(a, x, teacher_index, teacher_logits, temperature)
    return _forward(a, x, loss, lse, workspace, stream)


def linear_distill_backward(grad, x, w, teacher_index, teacher_logits, lse, *, temperature: float = 1.0,
                            b_layout: str = "nk", dx=None, dw=None, need_dx: bool = True, need_dw: bool = True,
                            accumulate_dw: bool = False, workspace=None, stream=None):
    """``(dx, dw)`` of ``linear_distill``; arguments as for ``linear_cross_entropy_backward``."""
    a = _product(x, w, b_layout)
    _distill(a, x, teacher_index, teacher_logits, temperature)
    return _backward(a, x, w, grad, lse, dx, dw, need_dx, need_dw, accumulate_dw, workspace, stream)
