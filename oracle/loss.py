"""fp64 reference of the vocabulary losses, with error bounds.

TEST INFRASTRUCTURE ONLY: imported by tests/, never by the library.  It shares
no code with the HIP path.  Plain numpy in float64 from the definitions:

    z = x . w^T,  lse = log sum_v exp(z_v / tau),  p = exp(z / tau - lse)
    xent:     loss = lse - z_y + zeta lse^2           dz = g ((1 + 2 zeta lse) p - onehot(y))
    distill:  q = softmax_K(s / tau)
              loss = tau^2 sum_k q_k (log q_k - z_{i_k} / tau + lse)     dz = g tau (p - sum_k q_k onehot(i_k))
    dx = dz . w,  dw = dz^T . x

Bounds (u: half a step of the operands' type, 2^-8 for bf16, 2^-11 for fp16;
f = 2^-24: half a step of fp32).  Each counts the roundings of a straightforward
fp32 evaluation, so it holds for any kernel that keeps fp32 throughout and
rounds dz and the results once:

* a logit is a chain of H / 16 matrix instructions, each of which rounds its sum
  of 16 products and the running value: |err z| <= ez = 2 (H / 16 + 8) f max_v sum_h |x||w|;
* log sum exp: the argument of each exponential is formed in fp32 from values up
  to max|z| / tau (relative error of the exponential 4 f max|z| / tau + 4 f), and
  no chain of additions is longer than 256 (a lane's 64 logits, then the tiles'
  sums): |err lse| <= ez / tau + (4 max|z| / tau + 260) f + f |lse|;
* the loss adds err(lse) and err(z), and a handful of roundings of its terms;
* dz: |err dz| <= u |dz| + |a| p (err z / tau + err lse + (4 max|z| / tau + 8) f) + 4 f (|a| p + |b| q),
  in fp16 also half its smallest step, 2^-25, over the scale that brings the
  largest |a| or |b| to at least 2^13.  A dz kept as the sum of two values of the
  type (`parts` = 2) rounds the first one's remainder, at most u |dz|, instead:
  u^2 |dz|;
* dx: sum_v err dz |w| + 2 (V / 16 + 8 + parts) f sum_v |dz||w| + u |dx|; dw
  alike over rows (`parts`: slices and pieces that are added up, at most 64); a
  result below the type's normal range is off by half its smallest step.
"""
from __future__ import annotations

from dataclasses import dataclass

import numpy as np

F32 = 2.0 ** -24
HALF_STEP = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": F32}
SMALLEST = {"bf16": 2.0 ** -134, "fp16": 2.0 ** -25, "fp32": 2.0 ** -150}   # half the smallest step
PARTS = 64


@dataclass
class Forward:
    loss: np.ndarray
    lse: np.ndarray
    loss_bound: np.ndarray
    lse_bound: np.ndarray
    z: np.ndarray
    z_bound: np.ndarray   # per row
    q: np.ndarray         # the target distribution [T,V]
    on: np.ndarray        # rows with a target
    bad: np.ndarray       # rows whose target is out of range


def _lse(z):
    m = z.max(axis=1, keepdims=True)
    m = np.where(np.isfinite(m), m, 0.0)
    return np.log(np.exp(z - m).sum(axis=1)) + m[:, 0]


def teacher(index, logits, tau, V):
    """(q [T,V], sum q log q, rows with entries, rows with an entry out of range)."""
    T, K = index.shape
    q = np.zeros((T, V))
    h = np.zeros(T)
    on = np.zeros(T, bool)
    bad = (index >= V).any(axis=1)
    for t in range(T):
        ks = [k for k in range(K) if 0 <= index[t, k] < V and logits[t, k] > -np.inf]
        if not ks:
            continue
        on[t] = True
        s = np.array([logits[t, k] / tau for k in ks])
        e = np.exp(s - s.max())
        qk = e / e.sum()
        for k, v in zip(ks, qk):
            q[t, index[t, k]] += v
            if v > 0:
                h[t] += v * np.log(v)
    return q, h, on, bad


def forward(x, w, dtype, target=None, index=None, logits=None, tau=1.0, zeta=0.0, ignore=-100, mutation=0) -> Forward:
    """x [T,H], w [V,H] float64 holding values of `dtype`.  `mutation` plants mistakes (for the tests of the tests)."""
    T, H = x.shape
    V = w.shape[0]
    z = x @ w.T
    ez = 2.0 * (H / 16 + 8) * F32 * (np.abs(x) @ np.abs(w).T).max(axis=1)
    lse = _lse(z / tau)
    top = np.abs(z).max(axis=1) / tau
    el = ez / tau + (4 * top + 260) * F32 + F32 * np.abs(lse)
    if target is not None:
        on = target != ignore
        bad = on & ((target < 0) | (target >= V))
        q = np.zeros((T, V))
        for t in range(T):
            if on[t] and not bad[t]:
                q[t, target[t]] = 1.0
        at = np.where(q > 0, z, 0.0).sum(axis=1)   # a logit of -infinity elsewhere takes no part
        loss = lse - at + (0.0 if mutation == 1 else zeta) * lse * lse
        bound = el + ez + 8 * F32 * (np.abs(lse) + 2 * top)
        if zeta:
            bound = bound + zeta * (2 * np.abs(lse) * el + 4 * F32 * lse * lse)
    else:
        q, h, on, bad = teacher(index, logits, 1.0 if mutation == 2 else tau, V)
        loss = tau * tau * (h - (q * z).sum(axis=1) / tau + lse)
        # the teacher's softmax: exponentials and sums of at most 1024 entries in
        # chains of 16 per lane and a tree, arguments up to the spread of s / tau
        spread = np.array([np.ptp(r[(i >= 0) & (r > -np.inf)]) if ((i >= 0) & (r > -np.inf)).any() else 0.0
                           for r, i in zip(logits, index)]) / tau
        eq = (4 * spread + 64 + 4 * np.abs(logits[np.isfinite(logits)]).max(initial=0.0) / tau) * F32
        bound = tau * tau * (el + ez / tau + 8 * F32 * (np.abs(lse) + 2 * top + np.abs(h)) +
                             eq * (2 + np.abs(h) + 2 * top + spread) + 200 * F32 * top)
    loss = np.where(on, loss, 0.0)
    loss[bad] = np.nan
    return Forward(loss, lse, np.where(on, bound, 0.0), el, z, ez, q, on, bad)


def backward(f: Forward, x, w, dtype, grad, tau=1.0, zeta=0.0, distill=False, dw_type=None, mutation=0, parts=1):
    """(dx, dw, bounds of both) with dw [V,H]; `parts`: values of `dtype` whose sum holds an entry of dz."""
    u, small = HALF_STEP[dtype], SMALLEST[dtype]
    T, H = x.shape
    V = w.shape[0]
    p = np.exp(f.z / tau - f.lse[:, None])
    g = np.where(f.on, grad, 0.0)
    a = (g * tau if distill else g * (1 + (1 if mutation == 3 else 2) * zeta * f.lse))[:, None]
    b = (g * tau if distill else g)[:, None]
    dz = a * p - b * (0.0 if mutation == 4 else 1.0) * f.q
    dz[~f.on] = 0.0
    top = np.abs(f.z).max(axis=1) / tau
    ep = (f.z_bound / tau + f.lse_bound + (4 * top + 8) * F32)[:, None]
    edz = u ** parts * np.abs(dz) + np.abs(a) * p * ep + (4 + 200 * distill) * F32 * (np.abs(a) * p + np.abs(b) * f.q)
    if dtype == "fp16":
        edz += 2.0 ** -25 * max(np.abs(a).max(initial=0), np.abs(b).max(initial=0)) / 2.0 ** 13
    dx, dw = dz @ w, dz.T @ x
    uw, sw = (u, small) if dw_type is None else (HALF_STEP[dw_type], SMALLEST[dw_type])
    bx = edz @ np.abs(w) + 2 * (V / 16 + 8 + PARTS) * F32 * (np.abs(dz) @ np.abs(w)) + u * np.abs(dx) + small
    bw = edz.T @ np.abs(x) + 2 * (T / 16 + 8 + PARTS) * F32 * (np.abs(dz).T @ np.abs(x)) + uw * np.abs(dw) + sw
    return dx, dw, bx, bw
