"""What an adapter holds reaches the rows that name it and no others: infinities and NaN in one
request's adapter leave every other request's results as they were, to the bit."""
import pytest
import torch

from lora_util import call_backward, call_forward, make

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
