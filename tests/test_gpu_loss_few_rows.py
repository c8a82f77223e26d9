"""GPU tests of the vocabulary losses' gradients for few rows, where no sum over many
rows averages the rounding of the logits' gradient: up to 64 rows it is kept in two
16-bit parts, so dx and dw are as good as results that are only rounded themselves."""
import numpy as np
import pytest
import torch

from oracle import loss as ol

from loss_util import call_backward, call_forward, f64, make, on_gpu, oracle_forward, ratio, say, to_layout

pytestmark = pytest.mark.gpu
KINDS = [("xent", 0, 1.0, 1e-3), ("distill", 7, 2.0, 0.0)]
SHAPES = [   # T, V, H, dtype, layout
    (1, 8, 8, "bf16", "nk"),
    (1, 5001, 264, "fp16", "nk"),
    (2, 20001, 136, "bf16", "nk"),
    (3, 3000, 1032, "bf16", "kn"),
    (16, 4097, 200, "fp16", "nk"),
    (31, 3001, 128, "bf16", "nk"),
    (32, 3000, 328, "fp16", "kn"),
    (33, 777, 72, "bf16", "nk"),
    (40, 100, 4096, "bf16", "nk"),
    (63, 16500, 136, "bf16", "nk"),
    (64, 5008, 520, "fp16", "kn"),
    (64, 5008, 520, "bf16", "kn"),
]


@pytest.fixture(scope="module")
def dg():
    import dense_gemm_work_amd as dg

    assert torch.cuda.is_available(), "GPU test run without a visible GPU"
    return dg


def inputs(shape, kind, seed=0):
    T, V, H, dtype, layout = shape
    name, K, tau, zeta = kind
    d = make(T, V, H, dtype, seed=seed + T + V, K=min(K, V), kind=name, ignored=0.1 if T > 8 else 0.0)
    return d, oracle_forward(d, dtype, tau, zeta)


def error(got, want):
    return float(np.linalg.norm(got - want) / np.linalg.norm(want))


@pytest.mark.parametrize("kind", KINDS, ids=lambda k: k[0])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_gradients_are_rounded_once(dg, shape, kind):
    T, V, H, dtype, layout = shape
    name, K, tau, zeta = kind
    d, f = inputs(shape, kind)
    g = on_gpu(d)
    say(f"  {name} {shape}")
    loss, lse = call_forward(dg, g, layout, tau, zeta)
    dx, dw = call_backward(dg, g, lse, layout, tau, zeta)
    d32 = torch.full(tuple(dw.shape), 7.0, device="cuda:0")
    call_backward(dg, g, lse, layout, tau, zeta, dw=d32, need_dx=False)
    args = (f, f64(d["x"]), f64(d["w"]), dtype, f64(d["grad"]), tau, zeta, name == "distill")
    rx, rw, bx, bw = ol.backward(*args, parts=2)
    _, _, _, b32 = ol.backward(*args, parts=2, dw_type="fp32")
    back = (lambda t: f64(t)) if layout == "nk" else (lambda t: f64(t).T)
    r = [ratio(f64(dx), rx, bx), ratio(back(dw), rw, bw), ratio(back(d32), rw, b32)]
    say(f"    worst ratios: dx {r[0]:.3f} dw {r[1]:.3f} fp32 dw {r[2]:.3f}; errors {error(f64(dx), rx):.6f} "
        f"{error(back(dw), rw):.6f} {error(back(d32), rw):.2e}")
    assert max(r) <= 1
    # a rounding is off by at most half a step, dz's by the square of that; beside them the
    # logits' own error, far below fp16's half step here
    u = ol.HALF_STEP[dtype]
    assert error(f64(dx), rx) <= u and error(back(dw), rw) <= u and error(back(d32), rw) <= max(u * u, 2.0 ** -16) * 2
    assert torch.equal(d32.to(dw.dtype), dw), "the 16-bit dw is the fp32 one, rounded"


@pytest.mark.parametrize("shape", [(2, 20001, 136, "bf16", "nk"), (40, 3000, 264, "fp16", "kn"), (64, 9001, 136, "bf16", "nk")], ids=str)
def test_the_same_bits_whatever_is_asked_for(dg, shape):
    # dx alone, dw alone (in more pieces of the vocabulary), both; fp32 and accumulated
    layout = shape[4]
    d, _ = inputs(shape, KINDS[0])
    g = on_gpu(d)
    loss, lse = call_forward(dg, g, layout)
    dx, dw = call_backward(dg, g, lse, layout)
    assert torch.equal(call_backward(dg, g, lse, layout, need_dw=False)[0], dx)
    assert torch.equal(call_backward(dg, g, lse, layout, need_dx=False)[1], dw)
    one = torch.full(tuple(dw.shape), 5.0, device="cuda:0")
    x1, _ = call_backward(dg, g, lse, layout, dw=one)
    assert torch.equal(x1, dx) and torch.equal(one.to(dw.dtype), dw)
    two = one.clone()
    call_backward(dg, g, lse, layout, dw=two, accumulate_dw=True)
    assert torch.equal(two, one + one)


def test_dw_alone_in_pieces(dg):
    # with few features the parts of dz are larger than what a slice of dx takes: pieces
    T, V, H = 64, 60001, 64
    plan = dg.gemm_loss_plan(dg.GemmLossArgs(T=T, V=V, H=H, layout=dg.GEMM_B_NK, dw=1), True, 256)
    assert plan.pieces > 3
    assert dg.gemm_loss_plan(dg.GemmLossArgs(T=T, V=V, H=H, layout=dg.GEMM_B_NK, dx=1, dw=1), True, 256).pieces == 1
    d = make(T, V, H, "bf16", seed=3)
    g = on_gpu(d)
    loss, lse = call_forward(dg, g)
    dx, dw = call_backward(dg, g, lse)
    assert torch.equal(call_backward(dg, g, lse, need_dx=False)[1], dw)
    one = torch.empty(V, H, device="cuda:0")
    call_backward(dg, g, lse, need_dx=False, dw=one)
    assert torch.equal(one.bfloat16(), dw)


@pytest.mark.parametrize("kind", KINDS, ids=lambda k: k[0])
@pytest.mark.parametrize("T", [3, 64])
def test_captured_and_replayed(dg, T, kind):
    V, H = 9001, 136
    name, K, tau, zeta = kind
    make_one = lambda seed: on_gpu(make(T, V, H, "fp16", K=K, kind=name, seed=seed, ignored=0.0))
    g = make_one(1)
    acc = torch.zeros(V, H, device="cuda:0")
    loss, lse = call_forward(dg, g, tau=tau, zeta=zeta)
    call_backward(dg, g, lse, tau=tau, zeta=zeta, dw=acc, accumulate_dw=True)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    say(f"  capture {name} T={T}")
    with torch.cuda.graph(graph):
        loss, lse = call_forward(dg, g, tau=tau, zeta=zeta)
        dx, dw = call_backward(dg, g, lse, tau=tau, zeta=zeta)
        call_backward(dg, g, lse, tau=tau, zeta=zeta, need_dx=False, dw=acc, accumulate_dw=True)
    want = torch.zeros_like(acc)
    acc.zero_()
    for r in range(4):
        for k, v in make_one(20 + r).items():
            g[k].copy_(v)
        for t in (loss, lse, dx, dw):
            t.fill_(7.0)
        say(f"  replay {r}")
        graph.replay()
        torch.cuda.synchronize()
        l2, e2 = call_forward(dg, g, tau=tau, zeta=zeta)
        x2, w2 = call_backward(dg, g, e2, tau=tau, zeta=zeta)
        call_backward(dg, g, e2, tau=tau, zeta=zeta, need_dx=False, dw=want, accumulate_dw=True)
        torch.cuda.synchronize()
        assert torch.equal(lse, e2) and torch.equal(dx, x2) and torch.equal(dw, w2) and torch.equal(acc, want)
    del graph


def test_rows_at_a_stride_keep_what_lies_between(dg):
    T, V, H = 64, 1000, 136
    d = on_gpu(make(T, V, H, seed=7))
    for layout in ("nk", "kn"):
        w = to_layout(d["w"], layout)
        loss, lse = call_forward(dg, d, layout)
        _, want = call_backward(dg, d, lse, layout, need_dx=False)
        rows, cols = w.shape
        for dtype, accumulate in ((torch.bfloat16, False), (torch.float32, False), (torch.float32, True)):
            full = torch.full((rows * (cols + 8) + 64,), 0.5, dtype=dtype, device="cuda:0")
            view = full[: rows * (cols + 8)].view(rows, cols + 8)
            call_backward(dg, d, lse, layout, need_dx=False, dw=view[:, :cols], accumulate_dw=accumulate)
            torch.cuda.synchronize()
            assert bool((view[:, cols:] == 0.5).all()) and bool((full[rows * (cols + 8):] == 0.5).all())
            got = view[:, :cols] - 0.5 if accumulate else view[:, :cols]
            if accumulate:   # one addition's rounding each way, of values below 1 and 0.5
                assert float((got - want.float()).abs().max()) <= float(want.float().abs().max()) * 2.0 ** -8 + 2.0 ** -23
            else:
                assert torch.equal(got.to(torch.bfloat16), want)
