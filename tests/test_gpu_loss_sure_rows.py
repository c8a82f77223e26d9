"""GPU tests of the vocabulary losses where the answer is (almost) certain: logits
in the hundreds whose row has all of its mass on the target.  Operands are small
integers, so every logit is exact whatever the order of its sum, and so are the
expected values: the maximum's own exponential is 1, the sum of exponentials at
least 1, a sure row's loss 0 and its gradient nothing but what the other entries
hold."""
import pytest
import torch

from loss_util import DTYPES, call_backward, call_forward, say, to_layout

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def dg():
    import dense_gemm_work_amd as dg

    assert torch.cuda.is_available(), "GPU test run without a visible GPU"
    return dg


SIZES = [   # T, V, H, dtype, layout: one per kind of logits tile
    (1, 1, 64, "bf16", "nk"),
    (40, 1, 64, "fp16", "nk"),
    (300, 1, 72, "bf16", "nk"),
    (3, 700, 64, "fp16", "nk"),          # 32 x 32
    (50, 16500, 136, "bf16", "nk"),      # 64 x 64
    (30, 3000, 136, "bf16", "kn"),       # 128 x 32
    (61, 3000, 136, "fp16", "kn"),       # 128 x 64
    (100, 9001, 136, "bf16", "nk"),      # 64 x 128
    (150, 20001, 136, "fp16", "nk"),     # 128 x 128
    (150, 20000, 136, "bf16", "kn"),
    (1000, 16001, 1016, "bf16", "nk"),   # 256 x 256
    (1000, 16000, 1016, "fp16", "kn"),
]


def sure(T, V, H, dtype, kind, layout):
    """Logits of a row: near m at the row's target, near -m elsewhere, m from 40 to 250."""
    g = torch.Generator().manual_seed(T + V)
    m = torch.randint(40, 251, (T,), generator=g).float()
    x = torch.zeros(T, H)
    x[:, 0] = m                                                           # bf16 holds integers to 256
    x[:, 2:8] = torch.randint(-1, 2, (T, 6), generator=g).float()
    w = torch.zeros(V, H)
    w[:, 0] = -1.0
    w[:, 2:8] = torch.randint(-1, 2, (V, 6), generator=g).float()
    y = V // 3
    w[y, 0] = 1.0
    x, w = x.to(DTYPES[dtype]), w.to(DTYPES[dtype])
    d = dict(x=x, w=w, grad=torch.rand(T, generator=g) + 0.5)
    target = torch.full((T,), y)
    if kind == "xent":
        d["target"] = target
    else:
        d["index"], d["logits"] = target[:, None].contiguous(), torch.randn(T, 1, generator=g)
    z = x.double() @ w.double()[y]
    d = {k: v.to(DEV) for k, v in d.items()}
    return d, z


@pytest.mark.parametrize("kind,tau", [("xent", 1.0), ("distill", 1.0), ("distill", 2.0), ("distill", 1.5)], ids=str)
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "x".join(map(str, s)))
def test_a_sure_rows_loss_is_zero(dg, size, kind, tau):
    T, V, H, dtype, layout = size
    d, z = sure(T, V, H, dtype, kind, layout)
    say(f"  {kind} {size} tau={tau}")
    loss, lse = call_forward(dg, d, layout, tau)
    # the other entries lie at least 2 (40 - 6) below, divided by tau <= 2: together at
    # most 16500 e^-34, which fp32 does not see beside 1
    worst = loss.abs().max().item()
    say(f"    loss in [{loss.min().item():.3e}, {loss.max().item():.3e}]")
    assert worst == 0.0
    # lse = m / tau: the division by tau as a product with its rounded inverse, two
    # roundings of half a step each
    assert float(((lse.double().cpu() - z / tau).abs() / (z / tau)).max()) <= 2 * 2.0 ** -24


@pytest.mark.parametrize("kind,tau", [("xent", 1.0), ("distill", 1.0), ("distill", 2.0)], ids=str)
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "x".join(map(str, s)))
def test_a_sure_rows_gradient_is_that_of_the_others(dg, size, kind, tau):
    # p of the target is exp(z - lse) with z = lse: 1, and dz there g - g = 0; the others
    # have p below e^-34, so |dx| <= 1.5 tau 16500 e^-34 max|w| < 1e-10 and
    # |dw| <= 1.5 tau T e^-34 256 < 1e-9
    T, V, H, dtype, layout = size
    d, z = sure(T, V, H, dtype, kind, layout)
    say(f"  {kind} {size} tau={tau}")
    loss, lse = call_forward(dg, d, layout, tau)
    dw = torch.full(tuple(to_layout(d["w"], layout).shape), 7.0, device=DEV)
    dx, dw = call_backward(dg, d, lse, layout, tau, dw=dw)
    say(f"    |dx| <= {dx.abs().max().item():.3e}, |dw| <= {dw.abs().max().item():.3e}")
    assert dx.abs().max().item() <= 1e-10 and dw.abs().max().item() <= 1e-9


@pytest.mark.parametrize("T,V", [(5, 900), (40, 20001), (300, 5003)], ids=str)
def test_losses_are_not_negative(dg, T, V):
    # lse >= the largest logit >= the target's, also after rounding: the difference is
    # exact at the maximum, the sum of exponentials at least 1, its logarithm at least 0
    g = torch.Generator().manual_seed(V)
    x = torch.randn(T, 128, generator=g) * 12.0
    w = torch.randn(V, 128, generator=g)
    x, w = x.bfloat16().to(DEV), w.bfloat16().to(DEV)
    target = (x.double() @ w.double().t()).argmax(1)
    loss, lse = dg.linear_cross_entropy(x, w, target)
    say(f"  {T} x {V}: loss from {loss.min().item():.3e}, lse to {lse.max().item():.0f}")
    assert lse.max().item() > 300 and loss.min().item() >= 0.0
