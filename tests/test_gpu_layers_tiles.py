"""GPU parity of the feed-forward block and the adapters on the kernel shapes that ordinary sizes take: the block's
gradients on every tile, the adapters in thin tiles whose k is sliced, rows beyond the first word of slabs.  Each case
asserts the plan (of 256 CUs) that it is there for; bounds and oracles are those of the other parity tests."""
import pytest
import torch

import ffn_util as fu
import lora_util as lu

pytestmark = pytest.mark.gpu
FFN = ("dx", "dw_gate", "dw_up", "dw_down")


@pytest.fixture(scope="module")
def dg():
    import dense_gemm_work_amd as dg

    assert torch.cuda.is_available(), "GPU test run without a visible GPU"
    return dg


BACKWARD = [   # T, H, F, dtype, act: tile of dg, du and h; of dx and whether its k is sliced; of dw and whether its rows are
    (999, 1032, 8200, "bf16", "gelu", 256, (128, True), (256, False)),
    (1001, 1544, 8200, "fp16", "silu", 256, (256, True), (256, False)),
    (3999, 1032, 2056, "bf16", "relu", 256, (256, True), (128, False)),
    (4999, 1032, 2056, "fp16", "gelu", 256, (128, False), (128, False)),
    (5001, 1544, 2056, "bf16", "silu", 256, (256, False), (256, False)),
    (7999, 1032, 1032, "fp16", "silu", 256, (256, False), (256, True)),
    (4999, 1544, 520, "bf16", "gelu", 128, (256, False), (128, True)),
    (131, 4104, 12296, "fp16", "relu", 128, (256, True), (128, False)),
    (4099, 136, 4000, "bf16", "silu", 128, (128, True), (256, True)),
    (1003, 136, 520, "fp16", "gelu", 128, (128, True), (128, True)),
]


@pytest.mark.parametrize("layout", ["nk", "kn"])
@pytest.mark.parametrize("case", BACKWARD, ids=lambda c: "x".join(map(str, c[:5])))
def test_ffn_backward_on_every_tile(dg, case, layout):
    T, H, F, dtype, act, first, out, dw = case
    p = dg.gemm_ffn_plan(dg.GemmFfnArgs(T=T, H=H, F=F, layout=dg.layout_word(layout, dtype), dx=1, dw_gate=1, dw_up=1, dw_down=1),
                         True, 256)
    assert (p.first_tile_f, p.first_tile_t) == (first, first)
    assert (p.out_tile_h, p.out_tile_t, p.out_splits > 1) == (out[0], out[0], out[1])
    assert (p.dw_tile_p, p.dw_tile_q, p.dw_splits > 1) == (dw[0], dw[0], dw[1])
    d = fu.make(T, H, F, dtype, seed=T, dev="cuda")
    got = fu.call_backward(dg, d, layout, act)
    want = fu.oracle_backward(d, act, dtype)
    worst = {n: fu.ratio(t if n == "dx" else fu.stored(t, layout), want[n]) for n, t in zip(FFN, got)}
    print("   ", {k: round(v, 3) for k, v in worst.items()}, flush=True)
    assert all(v <= 1 for v in worst.values()), worst
    # fp32 gradients, new and added to: the same sums, rounded to the type above
    new = [torch.full(tuple(t.shape), 7.0, device="cuda") for t in got[1:]]
    fu.call_backward(dg, d, layout, act, need_dx=False, **dict(zip(FFN[1:], new)))
    assert all(torch.equal(a.to(b.dtype), b) for a, b in zip(new, got[1:]))
    total = [torch.full_like(t, 0.5) for t in new]
    fu.call_backward(dg, d, layout, act, need_dx=False, accumulate_dw=True, **dict(zip(FFN[1:], total)))
    assert all(torch.equal(t, n + 0.5) for t, n in zip(total, new))


@pytest.mark.parametrize("layout", ["nk", "kn"])
@pytest.mark.parametrize("size", [(999, 1032, 8200), (5001, 1544, 2056), (131, 4104, 12296)], ids=str)
def test_ffn_two_strides_on_large_tiles(dg, size, layout):
    # w_gate's rows 8 elements further apart than w_up's: dx from two products through the slots
    T, H, F = size
    d = fu.make(T, H, F, "bf16", seed=T, dev="cuda")
    w = fu.stored(d["w_gate"], layout)
    wide = torch.full((w.shape[0], w.shape[1] + 8), float("nan"), dtype=w.dtype, device="cuda")
    wide[:, :-8] = w
    weights = wide[:, :-8], *(fu.stored(d[k], layout) for k in fu.WEIGHTS[1:])
    dx = dg.gated_ffn_backward(d["dy"], d["x"], *weights, d["gate"], d["up"], b_layout=layout, need_dw=False)[0]
    assert fu.ratio(dx, fu.oracle_backward(d, "silu", "bf16")["dx"]) <= 1


THIN = [   # T, H, N, L, R, dtype: what T * R elements a result cost the join keeps the adapters in the tiles:
    # 2 T R N / 8e6 us (backward: H) against 6 + L / 2, or ranks above 256, which the join does not take
    (20, 4104, 1032, 2, 320, "bf16"),     # 64 x 32, fewer adapters than slices: some have none
    (30, 1032, 1064, 9, 264, "fp16"),     # more adapters than slices
    (50, 1032, 1064, 9, 320, "bf16"),     # 64 x 64
    (64, 4104, 4096, 2, 1024, "fp16"),
    (100, 1032, 1064, 9, 264, "fp16"),    # 64 x 128
    (128, 4096, 8192, 4, 128, "bf16"),    # 34 (17) against 8
    (127, 2056, 2064, 3, 264, "bf16"),
]


@pytest.mark.parametrize("layout", ["nk", "kn"])
@pytest.mark.parametrize("order", ["mixed", "packed"])
@pytest.mark.parametrize("case", THIN, ids=lambda c: "x".join(map(str, c)))
def test_adapters_in_sliced_thin_tiles(dg, case, order, layout):
    T, H, N, L, R, dtype = case
    for backward in (False, True):
        a = dg.GemmLoraArgs(T=T, H=H, N=N, R=R, adapters=L, layout=dg.layout_word(layout, dtype), dx=1, da=1, db=1)
        p = dg.gemm_lora_plan(a, backward, 256)
        assert (p.out_tile_p, p.out_tile_t) == (64, 32 if T <= 32 else 64 if T <= 64 else 128)
        assert p.out_splits > 1 and p.out_whole == 0
        assert R > 256 or T * R * (H if backward else N) * 2 / 8e6 > 6 + L / 2
    d = lu.make(T, H, N, L, R, dtype, order, seed=T + R, dev="cuda")
    r = lu.ratio(lu.call_forward(dg, d, layout), lu.oracle_forward(d, dtype))
    got, want = lu.call_backward(dg, d, layout), lu.oracle_backward(d, dtype)
    worst = [r, lu.ratio(got[0], want["dx"]), *(lu.ratio(lu.stored(t, layout), want[k]) for k, t in zip(("da", "db"), got[1:]))]
    print("   ", [round(v, 3) for v in worst], flush=True)
    assert all(v <= 1 for v in worst), worst


@pytest.mark.parametrize("layout", ["nk", "kn"])
@pytest.mark.parametrize("case", [(4500, 2056, 4104, 6, 16, "bf16", 1), (9000, 2056, 4104, 4, 24, "fp16", 2)], ids=str)
def test_adapters_gradients_beyond_the_first_64_slabs(dg, case, layout):
    T, H, N, L, R, dtype, splits = case
    a = dg.GemmLoraArgs(T=T, H=H, N=N, R=R, adapters=L, layout=dg.layout_word(layout, dtype), da=1, db=1)
    assert dg.gemm_lora_plan(a, True, 256).dab_splits == splits and -(-T // 64) // splits > 64
    d = lu.make(T, H, N, L, R, dtype, "none", seed=T, dev="cuda")
    end = T // splits                             # of the first slice's rows, about
    d["adapter"][end - 100:end - 20] = 0          # its last slabs only
    d["adapter"][130:140] = 1                     # an early slab and the very last
    d["adapter"][T - 3:] = 1
    d["adapter"][64 * 64 - 1:64 * 64 + 2] = 2     # both sides of a word's end
    got = lu.call_backward(dg, d, layout, need_dx=False)
    want = lu.oracle_backward(d, dtype)
    worst = [lu.ratio(lu.stored(t, layout), want[k]) for k, t in zip(("da", "db"), got[1:])]
    print("   ", [round(v, 3) for v in worst], flush=True)
    assert all(v <= 1 for v in worst), worst
    assert int(torch.count_nonzero(got[1][3])) == 0 and int(torch.count_nonzero(got[2][3])) == 0
