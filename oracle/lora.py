"""64-bit reference of the projection with low-rank adapters, with error bounds.

TEST INFRASTRUCTURE ONLY: imported by tests/, never by the library.  It shares no
code with the HIP path.  Plain torch in float64, on the device of its arguments,
one adapter after the other, from the definitions (weights as stored for "nk"):

    s_t = c x_t . a[l]^T,   y_t = x_t . w^T + s_t . b[l]^T
    ds_t = c dy_t . b[l],   dx_t = dy_t . w + ds_t . a[l],   da[l] = sum ds_t (x) x_t,   db[l] = sum dy_t (x) s_t

Bounds (h: half a step of the operands' type, 2^-8 for bf16, 2^-11 for fp16;
f = 2^-24: half a step of fp32), each the roundings of a straightforward fp32
evaluation that rounds s, ds and the results once:

* a product over K is a chain of K / 16 matrix instructions, each of which rounds
  its sum of 16 products and the running value.  Cut into S slices of at least 128
  of K each, it is a chain of K / (16 S) and S sums, with S <= K / 128 never more
  than K / 16 + 8.  64 more cover the fixed parts: halves of a chain that are joined,
  eight products a lane and the lanes' sums where rows are multiplied one by one:
  2 (K / 16 + 8 + 64) f sum |a||b|.  Zeros from other rows or adapters add nothing;
  a row's sum passes one instruction pair more for each adapter of its tile, at
  most 256 of ranks of at most 64 slabs, that add zero and round nothing.
* s and ds: the product's error times |c|, 2 f for the scale, h for their rounding,
  half the type's smallest step below its normal range;
* y, dx, da and db: the operand's error through the product, both products' own,
  and one rounding.
"""
from __future__ import annotations

import torch

F32 = 2.0 ** -24
HALF_STEP = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": F32}
SMALLEST = {"bf16": 2.0 ** -134, "fp16": 2.0 ** -25, "fp32": 2.0 ** -150}   # half the smallest step
FIXED = 64


def product(a, b):
    """a . b and the bound of its fp32 evaluation's error."""
    return a @ b, 2.0 * (a.shape[1] / 16 + 8 + FIXED) * F32 * (a.abs() @ b.abs())


def narrow(x, factor, c, dtype):
    """c x . factor^T as the type holds it: value and bound."""
    v, e = product(x, factor.t())
    v = c * v
    return v, abs(c) * e + (2 * F32 + HALF_STEP[dtype]) * v.abs() + SMALLEST[dtype]


def forward(x, w, a, b, adapter, scale, dtype, mutation=0):
    """(y, bound).  `mutation` plants a mistake (for the tests of the tests)."""
    y, e = product(x, w.t())
    for i in range(a.shape[0]):
        rows = torch.nonzero(adapter == i)[:, 0]
        if not len(rows):
            continue
        c = 1.0 if scale is None or mutation == 1 else float(scale[i])
        s, es = narrow(x[rows], a[i], c, dtype)
        v, ev = product(s, b[i if mutation != 2 else 0].t())
        y[rows] += v
        e[rows] += ev + es @ b[i].t().abs()
    y[adapter >= a.shape[0]] = float("nan")
    return y, e + HALF_STEP[dtype] * y.abs().nan_to_num() + SMALLEST[dtype]


def backward(dy, x, w, a, b, adapter, scale, dtype, dab_type=None, mutation=0):
    """{name: (value, bound)} of dx, da and db."""
    h, small = HALF_STEP[dab_type or dtype], SMALLEST[dab_type or dtype]
    dx, ex = product(dy, w)
    out = {k: (torch.zeros_like(t), torch.full_like(t, small)) for k, t in (("da", a), ("db", b))}
    for i in range(a.shape[0]):
        rows = torch.nonzero(adapter == i)[:, 0]
        if not len(rows):
            continue
        c = 1.0 if scale is None else float(scale[i])
        s, es = narrow(x[rows], a[i], c, dtype)
        ds, eds = narrow(dy[rows], b[i].t(), c if mutation != 3 else 1.0, dtype)
        v, ev = product(ds, a[i])
        dx[rows] += v
        ex[rows] += ev + eds @ a[i].abs()
        for key, outs, e_outs, ins, e_ins in (("da", ds, eds, x[rows], None), ("db", dy[rows], None, s, es)):
            v, ev = product(outs.t(), ins)
            e = e_outs.t() @ ins.abs() if e_ins is None else outs.t().abs() @ e_ins
            out[key][0][i] = v
            out[key][1][i] = ev + e + h * v.abs() + small
    dx[adapter >= a.shape[0]] = float("nan")
    return dict(dx=(dx, ex + HALF_STEP[dtype] * dx.abs().nan_to_num() + SMALLEST[dtype]), **out)
