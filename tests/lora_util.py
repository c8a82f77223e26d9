"""Shared helpers of the adapters' tests: seeded inputs, calls, comparison with the 64-bit oracle."""
from __future__ import annotations

import math

import torch

from oracle import lora as orc

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def make(T, H, N, L, R, dtype="bf16", order="mixed", seed=0, dev="cpu"):
    """x, w, a, b as stored for "nk", dy, scale and the rows' adapters: "mixed" any order, "packed" requests one
    after the other, "one" a single adapter, "none"."""
    g = torch.Generator(device="cpu").manual_seed(seed)
    dt = DTYPES[dtype]

    def randn(*shape):
        return torch.randn(*shape, generator=g)

    d = {"x": randn(T, H).to(dt), "w": (randn(N, H) / math.sqrt(H)).to(dt), "a": (randn(L, R, H) / math.sqrt(H)).to(dt),
         "b": (randn(L, N, R) / math.sqrt(R)).to(dt), "dy": randn(T, N).to(dt), "scale": torch.rand(L, generator=g) + 0.5}
    if order == "mixed":
        d["adapter"] = torch.randint(-1, L, (T,), generator=g)
    elif order == "packed":
        d["adapter"] = torch.randint(-1, L, (T // 37 + 1,), generator=g).repeat_interleave(37)[:T].contiguous()
    else:
        d["adapter"] = torch.full((T,), L - 1 if order == "one" else -1)
    return {k: v.to(dev) for k, v in d.items()}


def stored(t, layout):
    return t if layout == "nk" else t.transpose(-1, -2).contiguous()


def args(d):
    return *(d[k].double() for k in ("x", "w", "a", "b")), d["adapter"], d["scale"]


def oracle_forward(d, dtype, **kw):
    return orc.forward(*args(d), dtype, **kw)


def oracle_backward(d, dtype, **kw):
    return orc.backward(d["dy"].double(), *args(d), dtype, **kw)


def call_forward(dg, d, layout="nk", **kw):
    return dg.linear_lora(d["x"], *(stored(d[k], layout) for k in ("w", "a", "b")), d["adapter"], scale=d["scale"],
                          b_layout=layout, **kw)


def call_backward(dg, d, layout="nk", **kw):
    return dg.linear_lora_backward(d["dy"], d["x"], *(stored(d[k], layout) for k in ("w", "a", "b")), d["adapter"],
                                   scale=d["scale"], b_layout=layout, **kw)


def ratio(got, want):
    """The worst |got - value| / bound; 0 where both are NaN."""
    value, bound = want
    if value.numel() == 0:
        return 0.0
    got = got.double()
    same = (got == value) | (got.isnan() & value.isnan())
    r = torch.where(same, 0.0, torch.nan_to_num((got - value).abs() / bound, nan=math.inf))
    return float(r.max())
