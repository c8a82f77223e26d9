"""GPU parity of the vocabulary losses (cross entropy and top-k distillation over
the logits of a product) with the fp64 oracle, every element within its bound."""
import numpy as np
import pytest
import torch

from oracle import loss as ol

from loss_util import call_backward, call_forward, f64, make, on_gpu, oracle_forward, ratio, say, to_layout

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dg():
    import dense_gemm_work_amd as dg

    assert torch.cuda.is_available(), "GPU test run without a visible GPU"
    return dg


SIZES = [   # T, V, H, dtype, layout
    (1, 8, 8, "bf16", "nk"),            # the smallest
    (1, 1, 64, "bf16", "nk"),           # a vocabulary of one entry
    (2, 257, 72, "fp16", "nk"),         # one entry behind a tile, ragged H
    (33, 1000, 128, "bf16", "kn"),
    (64, 4096, 256, "bf16", "nk"),
    (127, 129, 64, "fp16", "nk"),
    (129, 3001, 200, "bf16", "nk"),     # odd vocabulary, ragged everything
    (200, 520, 328, "fp16", "kn"),
    (256, 2048, 512, "bf16", "nk"),
    (300, 1111, 1024, "fp16", "nk"),
    (513, 776, 136, "bf16", "kn"),
    (1030, 640, 64, "bf16", "nk"),
]
KINDS = [("xent", 0, 1.0, 0.0), ("xent", 0, 1.0, 1e-3), ("distill", 1, 1.0, 0.0), ("distill", 7, 2.0, 0.0),
         ("distill", 33, 0.5, 0.0)]


@pytest.mark.parametrize("kind", KINDS, ids=lambda k: f"{k[0]}-K{k[1]}-tau{k[2]}-z{k[3]}")
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "x".join(map(str, s)))
def test_forward_and_backward(dg, size, kind):
    T, V, H, dtype, layout = size
    name, K, tau, zeta = kind
    K = min(K, V)
    d = make(T, V, H, dtype, seed=T + V, K=K, kind=name)
    f = oracle_forward(d, dtype, tau, zeta)
    g = on_gpu(d)
    say(f"  {name} T={T} V={V} H={H} {dtype} {layout} K={K} tau={tau} zeta={zeta}")
    loss, lse = call_forward(dg, g, layout, tau, zeta)
    torch.cuda.synchronize()
    assert ratio(f64(lse), f.lse, f.lse_bound) <= 1
    assert ratio(f64(loss), f.loss, f.loss_bound) <= 1
    assert torch.equal(loss.cpu()[torch.from_numpy(~f.on)], torch.zeros(int((~f.on).sum())))
    say("    backward")
    dx, dw = call_backward(dg, g, lse, layout, tau, zeta)
    torch.cuda.synchronize()
    rx, rw, bx, bw = ol.backward(f, f64(d["x"]), f64(d["w"]), dtype, f64(d["grad"]), tau, zeta, name == "distill")
    dwn = f64(dw) if layout == "nk" else f64(dw).T
    say(f"    worst ratios: dx {ratio(f64(dx), rx, bx):.3f} dw {ratio(dwn, rw, bw):.3f}")
    assert ratio(f64(dx), rx, bx) <= 1
    assert ratio(dwn, rw, bw) <= 1
    assert torch.equal(dx.cpu()[torch.from_numpy(~f.on)].float(), torch.zeros(int((~f.on).sum()), H))
