"""Shared helpers of the feed-forward block's tests: seeded inputs, calls, comparison with the 64-bit oracle."""
from __future__ import annotations

import math

import torch

from oracle import ffn as of

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
WEIGHTS = ("w_gate", "w_up", "w_down")


def make(T, H, F, dtype="bf16", seed=0, dev="cpu"):
    """x, the weights as stored for "nk", dy, and gate and up as a forward call keeps them."""
    g = torch.Generator(device="cpu").manual_seed(seed)
    dt = DTYPES[dtype]

    def randn(*shape):
        return torch.randn(*shape, generator=g)

    d = {"x": randn(T, H).to(dt), "w_gate": (randn(F, H) * (1.5 / math.sqrt(H))).to(dt), "w_up": (randn(F, H) / math.sqrt(H)).to(dt),
         "w_down": (randn(H, F) / math.sqrt(F)).to(dt), "dy": randn(T, H).to(dt)}
    d = {k: v.to(dev) for k, v in d.items()}
    x = d["x"].double()
    d["gate"], d["up"] = ((x @ d[w].double().t()).to(dt) for w in ("w_gate", "w_up"))
    return d


def stored(t, layout):
    return t if layout == "nk" else t.t().contiguous()


def doubles(d, *names):
    return [d[n].double() for n in names]


def oracle_forward(d, act, dtype, **kw):
    return of.forward(*doubles(d, "x", *WEIGHTS), act, dtype, parts=2 if d["x"].shape[0] <= 64 else 1, **kw)


def oracle_backward(d, act, dtype, **kw):
    return of.backward(*doubles(d, "dy", "x", *WEIGHTS, "gate", "up"), act, dtype,
                       parts=2 if d["x"].shape[0] <= 64 else 1, **kw)


def call_forward(dg, d, layout="nk", act="silu", **kw):
    return dg.gated_ffn(d["x"], *(stored(d[w], layout) for w in WEIGHTS), activation=act, b_layout=layout, **kw)


def call_backward(dg, d, layout="nk", act="silu", **kw):
    return dg.gated_ffn_backward(d["dy"], d["x"], *(stored(d[w], layout) for w in WEIGHTS), d["gate"], d["up"],
                                 activation=act, b_layout=layout, **kw)


def ratio(got, want):
    """The worst |got - value| / bound."""
    value, bound = want
    if value.numel() == 0:
        return 0.0
    r = (got.double() - value).abs() / bound
    return float(torch.where(got.double() == value, 0.0, torch.nan_to_num(r, nan=math.inf)).max())
