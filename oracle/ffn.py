"""64-bit reference of the gated feed-forward block, with error bounds.

TEST INFRASTRUCTURE ONLY: imported by tests/, never by the library.  It shares no
code with the HIP path.  Plain torch in float64, on the device of its arguments,
from the definitions (weights as stored for "nk"):

    g = x . w_gate^T,  u = x . w_up^T,  h = act(g) u,  y = h . w_down^T
    dh = dy . w_down,  dg = dh u act'(g),  du = dh act(g),  dx = dg . w_gate + du . w_up
    dw_gate = dg^T . x,  dw_up = du^T . x,  dw_down = dy^T . h

Bounds (s: half a step of the operands' type, 2^-8 for bf16, 2^-11 for fp16;
f = 2^-24: half a step of fp32; `parts`: values of the type whose sum holds h, dg
or du), each the roundings of a straightforward fp32 evaluation that rounds h, dg,
du and the results once:

* a product over K is a chain of K / 16 matrix instructions, each of which rounds
  its sum of 16 products and the running value.  Cut into S slices of at least 128
  of K each, it is a chain of K / (16 S) and S sums, with S <= K / 128 never more
  than K / 16 + 8.  64 more cover the fixed parts: halves of a chain that are joined,
  eight products a lane and the lanes' sums where rows are multiplied one by one:
  2 (K / 16 + 8 + 64) f sum |a||b|;
* act: silu's exponential has an argument of up to |g| log2 e, rounded twice (a
  relative error of 2 |g| f), and a handful of roundings follow: (8 + 2 |g|) f |act|,
  its slope (16 + 4 |g|) f; gelu's Phi is within 7.5e-8 (half the error of the
  approximation of erf) and 16 f (its polynomial's terms reach 1.5, its bell
  exp(-g^2 / 2) has a relative error of 2 g^2 f, and g^2 times the bell is at most
  0.74): |g| (7.5e-8 + 16 f), its slope, which adds g times the bell, 7.5e-8 + 32 f;
* |act'| is at most 1.13, so err act(g) <= 1.13 err g + that;
* h, dg and du: the products of their factors' errors, 4 f for their own
  multiplications, s^parts for their rounding, half the type's smallest step below
  its normal range;
* y, dx and the weights' gradients: the operand's error through the product, the
  product's own, and one rounding.
"""
from __future__ import annotations

import math

import torch

F32 = 2.0 ** -24
HALF_STEP = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": F32}
SMALLEST = {"bf16": 2.0 ** -134, "fp16": 2.0 ** -25, "fp32": 2.0 ** -150}   # half the smallest step
FIXED = 64
STEEPEST = 1.13   # the largest slope: gelu's, 1.1290


def product_error(a, b_t, K):
    """Bound of a . b_t accumulated in fp32."""
    return 2.0 * (K / 16 + 8 + FIXED) * F32 * (a.abs() @ b_t.abs())


def activation(g, act):
    """(act(g), act'(g), error of an fp32 evaluation of either)."""
    if act == "relu":
        return g.clamp(min=0), (g > 0).double(), torch.zeros_like(g), torch.zeros_like(g)
    if act == "silu":
        p = torch.sigmoid(g)
        a, s = g * p, p * (1 + g * (1 - p))
        return a, s, (8 + 2 * g.abs()) * F32 * a.abs(), (16 + 4 * g.abs()) * F32
    phi = 0.5 * torch.erfc(-g / math.sqrt(2))
    bell = torch.exp(-0.5 * g * g) / math.sqrt(2 * math.pi)
    return (g * phi, phi + g * bell, g.abs() * (7.5e-8 + 16 * F32), torch.full_like(g, 7.5e-8 + 32 * F32))


def forward(x, w_gate, w_up, w_down, act, dtype, parts=1, mutation=0):
    """{name: (value, bound)} of y, gate and up.  `mutation` plants a mistake (for the tests of the tests)."""
    s, small = HALF_STEP[dtype], SMALLEST[dtype]
    H, F = x.shape[1], w_gate.shape[0]
    g, u = x @ w_gate.t(), x @ w_up.t()
    eg, eu = product_error(x, w_gate.t(), H), product_error(x, w_up.t(), H)
    if mutation == 1:
        g, u = u, g
    a, _, ea, _ = activation(g, act)
    ea = ea + STEEPEST * eg
    h = a * u
    eh = u.abs() * ea + a.abs() * eu + ea * eu + (4 * F32 + s ** parts) * h.abs() + small
    y = h @ w_down.t()
    ey = eh @ w_down.t().abs() + product_error(h, w_down.t(), F) + s * y.abs() + small
    return {"y": (y, ey), "gate": (g, eg + s * g.abs() + small), "up": (u, eu + s * u.abs() + small)}


def backward(dy, x, w_gate, w_up, w_down, gate, up, act, dtype, dw_type=None, parts=1, mutation=0):
    """{name: (value, bound)} of dx, dw_gate, dw_up and dw_down."""
    s, small = HALF_STEP[dtype], SMALLEST[dtype]
    sw, smallw = (s, small) if dw_type is None else (HALF_STEP[dw_type], SMALLEST[dw_type])
    T, H = x.shape
    F = w_gate.shape[0]
    a, slope, ea, es = activation(gate, act)
    if mutation == 2:
        slope = torch.ones_like(slope)
    dh, edh = dy @ w_down, product_error(dy, w_down, H)
    dg, du, h = dh * up * slope, dh * a, a * up
    own = lambda v: (4 * F32 + s ** parts) * v.abs() + small   # noqa: E731
    edg = up.abs() * (slope.abs() * edh + (dh.abs() + edh) * es) + own(dg)
    edu = a.abs() * edh + (dh.abs() + edh) * ea + own(du)
    eh = up.abs() * ea + own(h)
    dx = dg @ w_gate + du @ w_up
    if mutation == 3:
        dx = dg @ w_gate
    edx = (edg @ w_gate.abs() + edu @ w_up.abs() + product_error(torch.cat((dg, du), 1), torch.cat((w_gate, w_up)), 2 * F) +
           s * dx.abs() + small)

    def grad(outs, e_outs, ins, e_ins):
        v = outs.t() @ ins
        e = e_outs.t() @ ins.abs() if e_outs is not None else outs.t().abs() @ e_ins
        return v, e + product_error(outs.t(), ins, T) + sw * v.abs() + smallw

    return {"dx": (dx, edx), "dw_gate": grad(dg, edg, x, None), "dw_up": grad(du, edu, x, None),
            "dw_down": grad(dy, None, h, eh)}
