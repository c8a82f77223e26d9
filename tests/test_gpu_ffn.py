"""GPU parity of the gated feed-forward block with the 64-bit oracle, every element within its bound."""
import pytest
import torch

from ffn_util import DTYPES, call_backward, call_forward, make, oracle_backward, oracle_forward, ratio, stored

pytestmark = pytest.mark.gpu
NAMES = ("dx", "dw_gate", "dw_up", "dw_down")


@pytest.fixture(scope="module")
def dg():
    import dense_gemm_work_amd as dg

    assert torch.cuda.is_available(), "GPU test run without a visible GPU"
    return dg


def check_forward(dg, d, layout, act, dtype, **kw):
    y, gate, up = call_forward(dg, d, layout, act, save=True, **kw)
    want = oracle_forward(d, act, dtype)
    got = dict(y=y, gate=gate, up=up)
    worst = {k: ratio(got[k], want[k]) for k in want}
    print("   ", {k: round(v, 3) for k, v in worst.items()}, flush=True)
    assert all(v <= 1 for v in worst.values()), worst
    # without the kept products: the same y
    assert torch.equal(call_forward(dg, d, layout, act, **kw).view(torch.int16), y.view(torch.int16))


def check_backward(dg, d, layout, act, dtype, **kw):
    got = call_backward(dg, d, layout, act, **kw)
    dw_type = "fp32" if got[1].dtype == torch.float32 else None
    want = oracle_backward(d, act, dtype, dw_type=dw_type)
    worst = {}
    for name, t in zip(NAMES, got):
        worst[name] = ratio(t if name == "dx" else stored(t, layout), want[name])
    print("   ", {k: round(v, 3) for k, v in worst.items()}, flush=True)
    assert all(v <= 1 for v in worst.values()), worst


SIZES = [   # T, H, F, dtype, layout, act
    (1, 8, 8, "bf16", "nk", "silu"),           # the smallest
    (1, 8, 8, "fp16", "kn", "gelu"),
    (1, 520, 4096, "bf16", "nk", "silu"),      # one token
    (2, 72, 264, "fp16", "nk", "relu"),        # ragged everything
    (3, 1032, 520, "bf16", "nk", "gelu"),
    (4, 4104, 72, "fp16", "nk", "silu"),       # the last by the kernels of single rows
    (5, 4104, 72, "bf16", "nk", "silu"),
    (31, 128, 1000, "bf16", "kn", "silu"),
    (33, 136, 8200, "fp16", "nk", "gelu"),     # 64 x 64 tiles
    (32, 64, 8216, "bf16", "nk", "silu"),      # many features, few rows
    (64, 256, 512, "bf16", "kn", "gelu"),      # the last with two parts
    (65, 256, 520, "bf16", "nk", "silu"),      # the first with one
    (65, 264, 512, "fp16", "kn", "relu"),
    (127, 200, 136, "fp16", "nk", "silu"),
    (300, 1032, 776, "bf16", "nk", "gelu"),
    (513, 136, 392, "fp16", "kn", "silu"),
    (1030, 640, 64, "bf16", "nk", "relu"),
]


@pytest.mark.parametrize("size", SIZES, ids=lambda s: "x".join(map(str, s)))
def test_forward(dg, size):
    T, H, F, dtype, layout, act = size
    check_forward(dg, make(T, H, F, dtype, seed=T + F, dev="cuda"), layout, act, dtype)


@pytest.mark.parametrize("size", SIZES, ids=lambda s: "x".join(map(str, s)))
def test_backward(dg, size):
    T, H, F, dtype, layout, act = size
    check_backward(dg, make(T, H, F, dtype, seed=T + F, dev="cuda"), layout, act, dtype)


# one case for each tile of each kernel (the plan's fields on 256 CUs)
SHAPES = [
    ("128x128", 200, 264, 4104, "bf16", "nk", dict(first_tile_f=64, first_tile_t=128)),
    ("128x128, kn", 200, 264, 4104, "fp16", "kn", dict(first_tile_f=64, first_tile_t=128)),
    ("256x256", 2000, 2056, 4000, "fp16", "nk", dict(first_tile_f=128, first_tile_t=256)),
    ("256x256, kn", 2000, 2056, 4000, "bf16", "kn", dict(first_tile_f=128, first_tile_t=256)),
]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: s[0])
def test_every_tile(dg, shape):
    _, T, H, F, dtype, layout, fields = shape
    plan = dg.gemm_ffn_plan(dg.GemmFfnArgs(T=T, H=H, F=F, layout=dg.layout_word(layout, dtype)), False, 256)
    for k, v in fields.items():
        assert getattr(plan, k) == v, (k, getattr(plan, k))
    d = make(T, H, F, dtype, seed=5, dev="cuda")
    check_forward(dg, d, layout, "silu", dtype)
    check_backward(dg, d, layout, "silu", dtype)
