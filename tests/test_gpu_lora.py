"""GPU parity of the projection with low-rank adapters with the 64-bit oracle, every element within its bound."""
import pytest
import torch

from lora_util import call_backward, call_forward, make, oracle_backward, oracle_forward, ratio, stored

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dg():
    import dense_gemm_work_amd as dg

    assert torch.cuda.is_available(), "GPU test run without a visible GPU"
    return dg


def check_forward(dg, d, layout, dtype, **kw):
    r = ratio(call_forward(dg, d, layout, **kw), oracle_forward(d, dtype))
    print(f"    y {r:.3f}", flush=True)
    assert r <= 1


def check_backward(dg, d, layout, dtype, **kw):
    got = call_backward(dg, d, layout, **kw)
    want = oracle_backward(d, dtype, dab_type="fp32" if got[1].dtype == torch.float32 else None)
    worst = {"dx": ratio(got[0], want["dx"])}
    for name, t in zip(("da", "db"), got[1:]):
        worst[name] = ratio(stored(t, layout), want[name])
    print("   ", {k: round(v, 3) for k, v in worst.items()}, flush=True)
    assert all(v <= 1 for v in worst.values()), worst


SIZES = [   # T, H, N, L, R, dtype, layout, order
    (1, 8, 8, 1, 8, "bf16", "nk", "one"),             # the smallest
    (1, 72, 136, 3, 8, "fp16", "kn", "one"),
    (1, 2048, 2048, 8, 16, "bf16", "nk", "one"),      # one token
    (1, 256, 256, 8, 16, "bf16", "nk", "none"),
    (2, 520, 264, 2, 24, "fp16", "nk", "mixed"),
    (3, 2056, 72, 3, 40, "bf16", "nk", "mixed"),
    (4, 264, 1032, 7, 256, "fp16", "nk", "mixed"),
    (5, 264, 1032, 7, 16, "bf16", "nk", "mixed"),
    (31, 264, 1000, 40, 16, "bf16", "kn", "mixed"),   # more adapters than rows
    (33, 128, 520, 5, 64, "bf16", "nk", "mixed"),
    (64, 1024, 264, 64, 8, "fp16", "nk", "mixed"),    # nearly a row each
    (96, 512, 1032, 64, 16, "bf16", "nk", "mixed"),
    (128, 200, 72, 4, 72, "bf16", "kn", "mixed"),     # a rank of two slabs
    (129, 200, 72, 3, 136, "fp16", "nk", "packed"),   # a rank of three
    (300, 136, 520, 7, 32, "bf16", "nk", "packed"),
    (300, 136, 520, 300, 8, "bf16", "kn", "mixed"),   # many adapters in every tile
    (777, 1032, 264, 5, 128, "fp16", "kn", "packed"),
    (1000, 64, 64, 1, 8, "bf16", "nk", "one"),        # one adapter, many rows
    (1030, 264, 2056, 9, 64, "bf16", "nk", "mixed"),
    (4100, 72, 136, 2, 16, "fp16", "kn", "packed"),   # more rows than one word's slabs
]


@pytest.mark.parametrize("size", SIZES, ids=lambda s: "x".join(map(str, s)))
def test_forward(dg, size):
    T, H, N, L, R, dtype, layout, order = size
    check_forward(dg, make(T, H, N, L, R, dtype, order, seed=T + N, dev="cuda"), layout, dtype)


@pytest.mark.parametrize("size", SIZES, ids=lambda s: "x".join(map(str, s)))
def test_backward(dg, size):
    T, H, N, L, R, dtype, layout, order = size
    check_backward(dg, make(T, H, N, L, R, dtype, order, seed=T + N, dev="cuda"), layout, dtype)


# one case for each tile of the wide product and each way its tiles are computed (the plan's fields on 256 CUs):
# all in slices, all whole, and whole but for the last ones
SHAPES = [   # T, H, N, R, dtype, backward, tile, how
    (20, 1032, 4104, 256, "bf16", False, (64, 32), "sliced"),
    (50, 1032, 4104, 128, "fp16", False, (64, 64), "sliced"),
    (100, 1032, 4104, 64, "bf16", False, (64, 128), "sliced"),
    (100, 136, 30000, 64, "fp16", False, (64, 128), "whole"),
    (1000, 2056, 1032, 16, "bf16", False, (128, 128), "sliced"),
    (1000, 1032, 8200, 16, "fp16", False, (128, 128), "tail"),
    (1000, 1032, 1032, 16, "bf16", True, (128, 128), "whole"),
    (4000, 2056, 1032, 16, "fp16", True, (128, 128), "tail"),
    (1000, 4096, 4104, 16, "bf16", False, (256, 256), "sliced"),
    (2000, 2056, 4096, 16, "fp16", True, (256, 256), "sliced"),
    (8192, 1032, 1032, 16, "bf16", False, (256, 256), "whole"),
    (5000, 2056, 4096, 72, "bf16", False, (256, 256), "tail"),
    (5000, 4096, 2056, 16, "fp16", True, (256, 256), "tail"),
]


@pytest.mark.parametrize("layout", ["nk", "kn"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"{s[6][0]}x{s[6][1]}-{s[7]}-{s[0]}x{s[1]}x{s[2]}-{'bwd' if s[5] else 'fwd'}")
def test_every_tile(dg, shape, layout):
    T, H, N, R, dtype, backward, tile, how = shape
    a = dg.GemmLoraArgs(T=T, H=H, N=N, R=R, adapters=6, layout=dg.layout_word(layout, dtype), dx=1, da=1, db=1)
    plan = dg.gemm_lora_plan(a, backward, 256)
    tiles = -(-(H if backward else N) // plan.out_tile_p) * -(-T // plan.out_tile_t)
    assert (plan.out_tile_p, plan.out_tile_t) == tile
    assert how == ("whole" if plan.out_whole == tiles else "tail" if plan.out_whole else "sliced")
    d = make(T, H, N, 6, R, dtype, "packed", seed=5, dev="cuda")
    (check_backward if backward else check_forward)(dg, d, layout, dtype)


EDGES = [   # T, H, N, L, R, dtype, layout, order: both sides of what few rows take, the largest rank
    (256, 264, 1032, 70, 16, "bf16", "nk", "mixed"),
    (257, 264, 1032, 70, 16, "bf16", "nk", "mixed"),
    (256, 264, 520, 300, 24, "fp16", "kn", "mixed"),
    (40, 136, 264, 40, 256, "bf16", "nk", "mixed"),
    (40, 136, 264, 40, 264, "bf16", "nk", "mixed"),
    (2, 136, 264, 2, 1024, "fp16", "nk", "mixed"),
    (60, 136, 264, 3, 1024, "bf16", "kn", "mixed"),
    (300, 264, 136, 3, 1024, "bf16", "nk", "mixed"),
    (5000, 1032, 2056, 5, 40, "bf16", "nk", "none"),      # large tiles without an adapter
]


@pytest.mark.parametrize("size", EDGES, ids=lambda s: "x".join(map(str, s)))
def test_edges(dg, size):
    T, H, N, L, R, dtype, layout, order = size
    d = make(T, H, N, L, R, dtype, order, seed=T + R, dev="cuda")
    check_forward(dg, d, layout, dtype)
    check_backward(dg, d, layout, dtype)


@pytest.mark.parametrize("layout", ["nk", "kn"])
@pytest.mark.parametrize("size", [(1, 4104, 72, 1, 8), (7, 72, 4104, 2, 32), (100, 520, 264, 25, 24), (256, 264, 1032, 64, 32)], ids=str)
def test_narrow_products_row_by_row(dg, size, layout):
    T, H, N, L, R = size
    for backward in (False, True):   # an adapter for every fourth row, ranks up to 32
        a = dg.GemmLoraArgs(T=T, H=H, N=N, R=R, adapters=L, layout=dg.layout_word(layout, "fp16"), dx=1, da=1, db=1)
        assert dg.gemm_lora_plan(a, backward, 256).low_tile_r == 8
        a.R = 40
        assert dg.gemm_lora_plan(a, backward, 256).low_tile_r > 8
    d = make(T, H, N, L, R, "fp16", "mixed", seed=T + R, dev="cuda")
    d["adapter"][T // 2] = -1 if T > 1 else 0
    check_forward(dg, d, layout, "fp16")
    check_backward(dg, d, layout, "fp16")
