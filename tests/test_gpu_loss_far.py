"""GPU tests of the vocabulary losses against bounds that are computed from the very
operands: offsets beyond 32 bits, and fp16 rows whose gradients differ by orders of
magnitude."""
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


def test_a_weight_of_more_than_2_to_the_32_bytes(dg):
    T, V, H, step = 4, 600000, 4096, 50000
    assert V * H > 1 << 31
    g = torch.Generator(device="cuda:0").manual_seed(5)
    x = torch.randn(T, H, generator=g, device="cuda:0").bfloat16()
    w = torch.empty(V, H, dtype=torch.bfloat16, device="cuda:0")
    w.normal_(generator=g).mul_(2.0 / 64)
    target = torch.tensor([1, V // 2 + 7, V - 1, V - 200], device="cuda:0")
    x64, rows = x.double(), torch.arange(T, device="cuda:0")
    # logits, and what their bound follows from: max over the vocabulary of sum_h |x||w|
    z, size = torch.empty(T, V, dtype=torch.float64, device="cuda:0"), torch.zeros(T, dtype=torch.float64, device="cuda:0")
    for i in range(0, V, step):
        part = w[i: i + step].double()
        z[:, i: i + step] = x64 @ part.t()
        size = torch.maximum(size, (x64.abs() @ part.abs().t()).amax(1))
    ez = 2 * (H / 16 + 8) * ol.F32 * size
    lse_want = torch.logsumexp(z, 1)
    top = z.abs().amax(1)
    el = ez + (4 * top + 260) * ol.F32 + ol.F32 * lse_want.abs()
    say(f"  sum |x||w| up to {size.max().item():.1f}, lse {lse_want.max().item():.2f}")
    loss, lse = dg.linear_cross_entropy(x, w, target)
    assert bool(((lse.double() - lse_want).abs() <= el).all())
    want = lse_want - z[rows, target]
    assert bool(((loss.double() - want).abs() <= el + ez + 8 * ol.F32 * (lse_want.abs() + 2 * top)).all())
    say("  backward")
    grad = torch.tensor([1.0, -0.5, 0.25, 2.0], device="cuda:0")
    dx, dw = dg.linear_cross_entropy_backward(grad, x, w, target, lse)
    p = torch.exp(z - lse_want[:, None])
    dz = p.clone()
    dz[rows, target] -= 1.0
    dz *= grad.double()[:, None]
    e = (ez + el + (4 * top + 8) * ol.F32)[:, None] * p + 4 * ol.F32 * p
    e[rows, target] += 4 * ol.F32
    e = 2.0 ** -8 * dz.abs() + e * grad.double().abs()[:, None]
    refx = torch.zeros(T, H, dtype=torch.float64, device="cuda:0")
    bx = torch.zeros_like(refx)
    for i in range(0, V, step):
        part, d = w[i: i + step].double(), dz[:, i: i + step]
        refx += d @ part
        bx += e[:, i: i + step] @ part.abs() + 2 * (V / 16 + 72) * ol.F32 * (d.abs() @ part.abs())
        refw = d.t().contiguous() @ x64
        bw = e[:, i: i + step].t().contiguous() @ x64.abs() + 2 * 73 * ol.F32 * (d.abs().t().contiguous() @ x64.abs())
        assert bool(((dw[i: i + step].double() - refw).abs() <= bw + 2.0 ** -8 * refw.abs() + 2.0 ** -134).all()), i
    assert bool(((dx.double() - refx).abs() <= bx + 2.0 ** -8 * refx.abs()).all())


@pytest.mark.parametrize("kind", [("xent", 0, 1.0, 1e-3), ("distill", 9, 2.0, 0.0)], ids=lambda k: k[0])
@pytest.mark.parametrize("shape", [(40, 3000, 136, "nk"), (130, 904, 64, "kn"), (600, 3000, 264, "nk")], ids=str)
def test_fp16_rows_whose_gradients_differ_by_orders_of_magnitude(dg, shape, kind):
    T, V, H, layout = shape
    name, K, tau, zeta = kind
    d = make(T, V, H, "fp16", seed=21, K=K, kind=name)
    d["grad"] = (d["grad"].abs() + 0.5) * 2.0 ** -torch.randint(0, 21, (T,), generator=torch.Generator().manual_seed(2))
    f = oracle_forward(d, "fp16", tau, zeta)
    g = on_gpu(d)
    loss, lse = call_forward(dg, g, layout, tau, zeta)
    dw = torch.empty(tuple(to_layout(g["w"], layout).shape), device="cuda:0")
    dx, _ = call_backward(dg, g, lse, layout, tau, zeta, dw=dw)
    args = (f, f64(d["x"]), f64(d["w"]), "fp16", f64(d["grad"]), tau, zeta, name == "distill")
    rx, _, bx, _ = ol.backward(*args)
    _, rw, _, bw = ol.backward(*args, dw_type="fp32")
    dwn = f64(dw) if layout == "nk" else f64(dw).T
    say(f"    {name} {shape}: worst ratios dx {ratio(f64(dx), rx, bx):.3f} dw {ratio(dwn, rw, bw):.3f}")
    assert ratio(f64(dx), rx, bx) <= 1 and ratio(dwn, rw, bw) <= 1
