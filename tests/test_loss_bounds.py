"""The oracle's bounds in fp16, without a GPU: a straightforward fp32 evaluation with
a scaled fp16 dz lies inside them, planted mistakes lie outside, and rows whose
gradients differ by orders of magnitude keep what the bounds promise."""
import numpy as np
import pytest
import torch

from oracle import loss as ol

from loss_util import f64, make, oracle_forward, ratio

CASES = [("xent", 0, 1.0, 0.0), ("xent", 0, 1.0, 1e-2), ("distill", 5, 2.0, 0.0), ("distill", 3, 0.5, 0.0)]


def evaluation(d, tau, zeta):
    """dx and dw in fp32 from a dz in fp16, scaled as the library scales it."""
    x, w, g = d["x"].float(), d["w"].float(), d["grad"]
    z = x @ w.t() / tau
    lse = torch.logsumexp(z, 1)
    if "target" in d:
        on = d["target"] >= 0
        q = torch.zeros_like(z)
        q[on, d["target"][on]] = 1.0
        a, b = g * (1 + 2 * zeta * lse), g
    else:
        on = (d["index"] >= 0).any(1)
        qk = torch.nan_to_num(torch.softmax(torch.where(d["index"] >= 0, d["logits"] / tau, -torch.inf), 1))
        q = torch.zeros(len(x), len(w) + 1).scatter_add_(1, torch.where(d["index"] < 0, len(w), d["index"]), qk)[:, :-1]
        a = b = g * tau
    a, b = torch.where(on, a, 0.0), torch.where(on, b, 0.0)
    scale = 2.0 ** (13 - np.floor(np.log2(max(a.abs().max().item(), b.abs().max().item()))))
    dz = a[:, None] * scale * torch.exp(z - lse[:, None]) - b[:, None] * scale * q
    dz = torch.where(on[:, None], dz, 0.0).half()
    assert torch.isfinite(dz).all() and dz.abs().max() <= 2.0 ** 14
    dz = dz.float()
    return (dz @ w / scale).half(), (dz.t() @ x / scale).half()


@pytest.mark.parametrize("spread", [0, 20], ids=["alike", "apart"])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_fp16_bounds_hold_and_have_teeth(case, spread):
    kind, K, tau, zeta = case
    d = make(120, 700, 64, "fp16", kind=kind, K=K, seed=5)
    d["grad"] = (d["grad"].abs() + 0.5) * 2.0 ** -torch.randint(0, spread + 1, (120,), generator=torch.Generator().manual_seed(1))
    f = oracle_forward(d, "fp16", tau, zeta)
    dx, dw = evaluation(d, tau, zeta)
    x, w, g = f64(d["x"]), f64(d["w"]), f64(d["grad"])
    rx, rw, bx, bw = ol.backward(f, x, w, "fp16", g, tau, zeta, kind == "distill")
    assert ratio(f64(dx), rx, bx) <= 1 and ratio(f64(dw), rw, bw) <= 1
    mx, mw, _, _ = ol.backward(f, x, w, "fp16", g, tau, zeta, kind == "distill", mutation=4)
    assert ratio(f64(dx), mx, bx) > 1 and ratio(f64(dw), mw, bw) > 1
    if zeta:
        mx, _, _, _ = ol.backward(f, x, w, "fp16", g, tau, zeta, mutation=3)
        assert ratio(f64(dx), mx, bx) > 1
