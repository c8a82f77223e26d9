"""What an adapter holds reaches the rows that name it and no others: infinities and NaN in one
request's adapter leave every other request's results as they were, to the bit."""
import pytest
import torch

from lora_util import call_backward, call_forward, make, oracle_backward, oracle_forward, ratio

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dg():
    import dense_gemm_work_amd as dg

    assert torch.cuda.is_available(), "GPU test run without a visible GPU"
    return dg


def bits(t):
    return t.view(torch.int16)


SIZES = [   # T, H, N, L, R, dtype, order: the tiles' sizes and the few rows' join, several adapters a tile
    (4, 72, 136, 3, 8, "bf16", "mixed"),
    (20, 136, 264, 3, 16, "fp16", "mixed"),
    (30, 136, 264, 4, 320, "bf16", "mixed"),      # too high a rank for the join: 64 x 32 tiles
    (60, 136, 264, 4, 320, "fp16", "mixed"),      # 64 x 64
    (128, 200, 72, 4, 72, "bf16", "mixed"),
    (128, 200, 264, 4, 320, "bf16", "mixed"),     # 64 x 128
    (300, 136, 520, 7, 32, "fp16", "mixed"),      # 128 x 128
    (1000, 264, 520, 9, 72, "bf16", "packed"),
    (5000, 2056, 2056, 5, 16, "bf16", "packed"),  # 256 x 256
    (5000, 1032, 2056, 5, 40, "fp16", "mixed"),
]


@pytest.mark.parametrize("layout", ["nk", "kn"])
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "x".join(map(str, s)))
def test_an_adapter_reaches_its_own_rows_alone(dg, size, layout):
    T, H, N, L, R, dtype, order = size
    d = make(T, H, N, L, R, dtype, order, seed=T + R, dev="cuda")
    d["adapter"][:3] = torch.tensor([0, 1, 2], device="cuda")
    y, (dx, da, db) = call_forward(dg, d, layout), call_backward(dg, d, layout)
    other = d["adapter"] != 1
    for value in (float("inf"), float("nan")):
        e = dict(d, a=d["a"].clone(), b=d["b"].clone())
        e["a"][1, R - 1, 5] = e["b"][1, N - 1, 3] = value
        got, (gx, ga, gb) = call_forward(dg, e, layout), call_backward(dg, e, layout)
        assert torch.equal(bits(got[other]), bits(y[other]))
        assert torch.equal(bits(gx[other]), bits(dx[other]))
        for l in range(L):
            if l != 1:
                assert torch.equal(bits(ga[l]), bits(da[l])) and torch.equal(bits(gb[l]), bits(db[l]))
        # its own: s, and so y and db, meet a's value; ds, and so dx and da, meet b's
        assert not bool(got[~other].isfinite().all()) and not bool(gx[~other].isfinite().all())
        assert not bool(ga[1].isfinite().all()) and not bool(gb[1].isfinite().all())


@pytest.mark.parametrize("layout", ["nk", "kn"])
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "x".join(map(str, s)))
def test_its_own_rows_are_the_definitions(dg, size, layout):
    # b's infinity is one result of each row that names its adapter, a's one of each row's gradient: these are
    # infinite with the definition's sign (NaN where it meets a zero), the others within their bounds
    T, H, N, L, R, dtype, order = size
    d = make(T, H, N, L, R, dtype, order, seed=T + R, dev="cuda")
    d["adapter"][:3] = torch.tensor([0, 1, 2], device="cuda")
    inf = float("inf")
    e = dict(d, b=d["b"].clone())
    e["b"][1, N - 1, R - 3], e["b"][2, 7, 0] = inf, -inf
    want = oracle_forward(e, dtype)
    assert int(want[0].isinf().sum()) >= 2 and ratio(call_forward(dg, e, layout), want) <= 1
    e = dict(d, a=d["a"].clone())
    e["a"][1, R - 3, H - 1], e["a"][2, 0, 7] = inf, -inf
    want = oracle_backward(e, dtype)["dx"]
    assert int(want[0].isinf().sum()) >= 2 and ratio(call_backward(dg, e, layout)[0], want) <= 1


@pytest.mark.parametrize("size", SIZES, ids=lambda s: "x".join(map(str, s)))
def test_a_broken_scale_stays_with_its_adapter(dg, size):
    T, H, N, L, R, dtype, order = size
    d = make(T, H, N, L, R, dtype, order, seed=T + R, dev="cuda")
    d["adapter"][:3] = torch.tensor([0, 1, 2], device="cuda")
    y, (dx, da, db) = call_forward(dg, d), call_backward(dg, d)
    other, rest = d["adapter"] != 1, [l for l in range(L) if l != 1]
    d["scale"][1] = float("nan")
    got, (gx, ga, gb) = call_forward(dg, d), call_backward(dg, d)
    for a, b in ((got[other], y[other]), (gx[other], dx[other]), (ga[rest], da[rest]), (gb[rest], db[rest])):
        assert torch.equal(bits(a), bits(b))
    assert all(bool(t.isnan().all()) for t in (got[~other], gx[~other], ga[1], gb[1]))
