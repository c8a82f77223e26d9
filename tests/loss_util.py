"""Shared helpers of the vocabulary-loss tests: seeded inputs and comparison with the fp64 oracle."""
from __future__ import annotations

import numpy as np
import torch

from oracle import loss as ol

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def say(*a):
    print(*a, flush=True)


def make(T, V, H, dtype="bf16", seed=0, spread=2.0, K=0, ignored=0.1, kind="xent"):
    """CPU tensors: x [T,H], w [V,H] in `dtype`; targets or teacher entries; grad."""
    rng = np.random.default_rng(seed)
    dt = DTYPES[dtype]
    x = torch.from_numpy(rng.standard_normal((T, H))).to(dt)
    w = torch.from_numpy(rng.standard_normal((V, H)) * spread / np.sqrt(H)).to(dt)
    d = dict(x=x, w=w, grad=torch.from_numpy(rng.uniform(-0.5, 1.5, T)).float())
    target = torch.from_numpy(rng.integers(0, V, T))
    if kind == "xent":
        target[torch.from_numpy(rng.random(T) < ignored)] = -100
        d["target"] = target
    else:
        index = np.stack([rng.permutation(V)[:K] if K <= V else rng.integers(0, V, K) for _ in range(T)]) if T else \
            np.zeros((0, K), np.int64)
        logits = rng.standard_normal((T, K)) * 3.0
        for t in range(T):
            r = rng.random()
            if r < ignored:
                index[t] = -1                                    # a row without entries
            elif r < 2 * ignored:
                index[t, rng.random(K) < 0.5] = -1               # padding among the entries
        d["index"] = torch.from_numpy(index.astype(np.int64))
        d["logits"] = torch.from_numpy(logits).float()
    return d


def f64(t):
    return t.double().cpu().numpy()


def to_layout(w, layout):
    return w if layout == "nk" else w.t().contiguous()


def ratio(got, want, bound):
    """The worst |got - want| / bound; 0 where both are the same NaN or infinity."""
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    same = (np.isnan(got) & np.isnan(want)) | (got == want)
    with np.errstate(invalid="ignore", divide="ignore"):
        r = np.abs(got - want) / bound
    r = np.where(same, 0.0, np.where(np.isfinite(r), r, np.inf))
    return float(r.max(initial=0.0))


def oracle_forward(d, dtype, tau=1.0, zeta=0.0, ignore=-100):
    if "target" in d:
        return ol.forward(f64(d["x"]), f64(d["w"]), dtype, target=d["target"].cpu().numpy(), zeta=zeta, ignore=ignore)
    return ol.forward(f64(d["x"]), f64(d["w"]), dtype, index=d["index"].cpu().numpy(), logits=f64(d["logits"]), tau=tau)


def call_forward(dg, d, layout="nk", tau=1.0, zeta=0.0, ignore=-100, w=None, **kw):
    w = to_layout(d["w"], layout) if w is None else w
    if "target" in d:
        return dg.linear_cross_entropy(d["x"], w, d["target"], b_layout=layout, z_loss=zeta, ignore_index=ignore, **kw)
    return dg.linear_distill(d["x"], w, d["index"], d["logits"], temperature=tau, b_layout=layout, **kw)


def call_backward(dg, d, lse, layout="nk", tau=1.0, zeta=0.0, ignore=-100, w=None, **kw):
    w = to_layout(d["w"], layout) if w is None else w
    if "target" in d:
        return dg.linear_cross_entropy_backward(d["grad"], d["x"], w, d["target"], lse, b_layout=layout, z_loss=zeta,
                                                ignore_index=ignore, **kw)
    return dg.linear_distill_backward(d["grad"], d["x"], w, d["index"], d["logits"], lse, temperature=tau,
                                      b_layout=layout, **kw)


def on_gpu(d, dev="cuda:0"):
    return {k: v.to(dev) for k, v in d.items()}
