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


# One case per kernel shape: the thin tiles, 64 x 128, 128 x 128, 256 x 256 with and
# without slices, the persistent dw, every storage.  (plan fields checked on 256 CUs)
SHAPES = [
    ("thin 32x32", 3, 4100, 520, "bf16", "nk", dict(tile_v=32, tile_t=32)),
    ("thin 64x64", 50, 16500, 136, "fp16", "nk", dict(tile_v=64, tile_t=64)),
    ("thin 64x64, few rows", 9, 20001, 264, "bf16", "nk", dict(tile_v=64, tile_t=64, dx_tile_t=32)),
    ("thin 128x32", 32, 3000, 328, "bf16", "kn", dict(tile_v=128, tile_t=32)),
    ("thin 128x64", 61, 5008, 136, "fp16", "kn", dict(tile_v=128, tile_t=64)),
    ("64x128", 100, 9001, 136, "bf16", "nk", dict(tile_v=64, tile_t=128)),
    ("128x128", 150, 20001, 136, "fp16", "nk", dict(tile_v=128, tile_t=128, dw_tile_p=128)),
    ("128x128 kn", 150, 20000, 136, "bf16", "kn", dict(tile_v=128, tile_t=128)),
    ("256x256", 1000, 16001, 1016, "bf16", "nk", dict(tile_v=256, tile_t=256, dw_tile_p=256)),
    ("256x256 kn", 1000, 16000, 1016, "fp16", "kn", dict(tile_v=256, tile_t=256, dw_tile_p=256)),
    ("256x256 dx", 2000, 16001, 2040, "bf16", "nk", dict(tile_v=256, dx_tile_h=256, dx_splits=4)),
    ("256x256 dx, kn", 2000, 16000, 2040, "bf16", "kn", dict(tile_v=256, dx_tile_h=256, dx_splits=4)),
    ("dw in slices", 3000, 300, 136, "bf16", "nk", dict()),
    ("dw in slices, kn", 3000, 296, 136, "fp16", "kn", dict()),
    ("short vocabulary, long rows", 40, 100, 4096, "bf16", "nk", dict()),
    ("one slab", 300, 3000, 8, "bf16", "nk", dict()),
    ("one whole slab", 300, 3000, 64, "fp16", "kn", dict()),
    ("two slabs, the second of 8", 700, 3000, 72, "fp16", "nk", dict()),
    ("one slab, few rows", 20, 3001, 40, "bf16", "nk", dict()),
    ("three slabs, few rows", 20, 3000, 136, "bf16", "kn", dict()),
]


@pytest.mark.parametrize("kind", [("xent", 0, 1.0, 1e-3), ("distill", 20, 2.0, 0.0)], ids=lambda k: k[0])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: s[0])
def test_every_kernel_shape(dg, shape, kind):
    what, T, V, H, dtype, layout, fields = shape
    name, K, tau, zeta = kind
    a = dg.GemmLossArgs(T=T, V=V, H=H, layout=dg.layout_word(layout, dtype), kind=int(K > 0), entries=K, dx=1, dw=1)
    plan = dg.gemm_loss_plan(a, True, 256)
    for k, v in fields.items():
        assert getattr(plan, k) == v, (what, k, getattr(plan, k))
    if what.startswith("dw in slices"):
        assert plan.dw_splits > 1
    d = make(T, V, H, dtype, seed=T + V, K=K, kind=name)
    f = oracle_forward(d, dtype, tau, zeta)
    g = on_gpu(d)
    say(f"  {what}: {name}")
    loss, lse = call_forward(dg, g, layout, tau, zeta)
    torch.cuda.synchronize()
    assert ratio(f64(lse), f.lse, f.lse_bound) <= 1
    assert ratio(f64(loss), f.loss, f.loss_bound) <= 1
    dx, dw = call_backward(dg, g, lse, layout, tau, zeta)
    torch.cuda.synchronize()
    rx, rw, bx, bw = ol.backward(f, f64(d["x"]), f64(d["w"]), dtype, f64(d["grad"]), tau, zeta, name == "distill")
    dwn = f64(dw) if layout == "nk" else f64(dw).T
    say(f"    worst ratios: loss {ratio(f64(loss), f.loss, f.loss_bound):.3f} dx {ratio(f64(dx), rx, bx):.3f} dw {ratio(dwn, rw, bw):.3f}")
    assert ratio(f64(dx), rx, bx) <= 1
    assert ratio(dwn, rw, bw) <= 1


def test_several_pieces_of_the_vocabulary(dg):
    # 65536 rows: pieces of 2048 entries, the last one ragged; dx is the sum over them
    T, V, H, dtype = 65536, 4503, 64, "bf16"
    plan = dg.gemm_loss_plan(dg.GemmLossArgs(T=T, V=V, H=H, layout=dg.GEMM_B_NK, dx=1, dw=1), True, 256)
    assert plan.pieces == 3 and plan.piece == 2048
    d = make(T, V, H, dtype, seed=1)
    g = on_gpu(d)
    say(f"  {T} x {V} x {H} in {plan.pieces} pieces")
    loss, lse = call_forward(dg, g)
    dx, dw = call_backward(dg, g, lse)
    torch.cuda.synchronize()
    x, w, grad, loss, lse, dx, dw = (f64(t) for t in (d["x"], d["w"], d["grad"], loss, lse, dx, dw))
    rw, bw = np.zeros((V, H)), np.zeros((V, H))
    for lo in range(0, T, 8192):
        s = slice(lo, lo + 8192)
        f = ol.forward(x[s], w, dtype, target=d["target"].numpy()[s])
        rx, pw, bx, pb = ol.backward(f, x[s], w, dtype, grad[s])
        assert ratio(loss[s], f.loss, f.loss_bound) <= 1 and ratio(lse[s], f.lse, f.lse_bound) <= 1
        assert ratio(dx[s], rx, bx) <= 1
        rw += pw
        bw += pb   # covers the whole: |dw| <= the sum of the parts' |dw|
        say(f"    rows to {lo + 8192}")
    # a row's part of the vocabulary is accumulated over all T rows, not 8192
    bw += 2 * (T / 16) * ol.F32 * np.abs(rw)
    assert ratio(dw, rw, bw) <= 1


def guarded(rows, cols, ld, dtype, dev="cuda:0"):
    """A [rows, cols] view with row stride ld inside a buffer of 7s."""
    full = torch.full((rows * ld + 64,), 7.0, dtype=dtype, device=dev)
    return full, full[: rows * ld].view(rows, ld)[:, :cols]


def guards_hold(full, view, ld):
    rows, cols = view.shape
    body = full[: rows * ld].view(rows, ld)
    return bool((body[:, cols:] == 7.0).all()) and bool((full[rows * ld:] == 7.0).all())


@pytest.mark.parametrize("layout", ["nk", "kn"])
@pytest.mark.parametrize("T", [5, 100, 700], ids=lambda t: f"T{t}")
def test_rows_at_a_stride(dg, T, layout):
    V, H, dtype = 1000, 136, "bf16"
    d = make(T, V, H, dtype, seed=7)
    f = oracle_forward(d, dtype)
    g = on_gpu(d)
    wl = to_layout(g["w"], layout)
    bx_, x = guarded(T, H, H + 24, torch.bfloat16)
    bw_, w = guarded(*wl.shape, wl.shape[1] + 40, torch.bfloat16)
    x.copy_(g["x"])
    w.copy_(wl)
    fx, dx = guarded(T, H, H + 8, torch.bfloat16)
    fw, dw = guarded(*wl.shape, wl.shape[1] + 16, torch.bfloat16)
    g["x"] = x
    say(f"  strided rows T={T} {layout}")
    loss, lse = call_forward(dg, g, layout, w=w)
    got = call_backward(dg, g, lse, layout, w=w, dx=dx, dw=dw)
    torch.cuda.synchronize()
    assert got[0] is dx and got[1] is dw
    assert guards_hold(fx, dx, H + 8) and guards_hold(fw, dw, wl.shape[1] + 16)
    assert guards_hold(bx_, x, H + 24) and guards_hold(bw_, w, wl.shape[1] + 40)
    rx, rw, bx, bw = ol.backward(f, f64(d["x"]), f64(d["w"]), dtype, f64(d["grad"]))
    assert ratio(f64(loss), f.loss, f.loss_bound) <= 1
    assert ratio(f64(dx), rx, bx) <= 1
    assert ratio(f64(dw) if layout == "nk" else f64(dw).T, rw, bw) <= 1


@pytest.mark.parametrize("shape", [(40, 3000, 264), (900, 2000, 264), (3000, 300, 136)], ids=str)
@pytest.mark.parametrize("layout", ["nk", "kn"])
def test_fp32_dw_and_accumulation(dg, shape, layout):
    T, V, H = shape
    V = V // 8 * 8
    d = make(T, V, H, "bf16", seed=8)
    g = on_gpu(d)
    say(f"  fp32 dw {shape} {layout}")
    loss, lse = call_forward(dg, g, layout)
    dw16 = call_backward(dg, g, lse, layout, need_dx=False)[1]
    wl = to_layout(g["w"], layout)
    dw = torch.full(wl.shape, 3.0, dtype=torch.float32, device="cuda:0")
    dx, got = call_backward(dg, g, lse, layout, need_dx=False, dw=dw)
    assert dx is None and got is dw
    torch.cuda.synchronize()
    f = oracle_forward(d, "bf16")
    _, rw, _, bw = ol.backward(f, f64(d["x"]), f64(d["w"]), "bf16", f64(d["grad"]), dw_type="fp32")
    back = (lambda t: f64(t)) if layout == "nk" else (lambda t: f64(t).T)
    assert ratio(back(dw), rw, bw) <= 1
    assert torch.equal(dw.to(torch.bfloat16), dw16), "the 16-bit dw is the fp32 one, rounded"
    twice = dw.clone()
    call_backward(dg, g, lse, layout, need_dx=False, dw=twice, accumulate_dw=True)
    torch.cuda.synchronize()
    assert torch.equal(twice, dw + dw)
    dx2, none = call_backward(dg, g, lse, layout, need_dw=False)
    assert none is None
    assert torch.equal(dx2, call_backward(dg, g, lse, layout)[0])


def test_refused_tensor_arguments(dg):
    d = on_gpu(make(16, 64, 32))
    loss, lse = call_forward(dg, d)
    x, w, t = d["x"], d["w"], d["target"]
    with pytest.raises(TypeError):
        dg.linear_cross_entropy(x, w, t.int())
    with pytest.raises(ValueError):
        dg.linear_cross_entropy(x, w, t[:-1])
    with pytest.raises(ValueError):
        dg.linear_cross_entropy(x, w, t.cpu())
    with pytest.raises(ValueError):
        dg.linear_cross_entropy(x, w.cpu(), t)
    with pytest.raises(ValueError):
        dg.linear_cross_entropy(x, w, t, b_layout="tn")
    with pytest.raises(ValueError):
        dg.linear_cross_entropy(x, w, t, b_layout="kn")           # w is [V,H]
    with pytest.raises(ValueError):
        dg.linear_cross_entropy(x.t().contiguous().t(), w, t)      # columns, not rows, contiguous
    with pytest.raises(ValueError):
        dg.linear_cross_entropy(x[:1].expand(16, 32), w, t)        # rows overlap
    with pytest.raises(dg.GemmError):
        dg.linear_cross_entropy(x, w, t, z_loss=-1.0)
    with pytest.raises(dg.GemmError):
        dg.linear_cross_entropy(x, w, t, workspace=torch.empty(256, dtype=torch.uint8, device="cuda:0"))
    with pytest.raises(dg.GemmError):
        dg.linear_distill(x, w, t[:, None], torch.zeros(16, 1, device="cuda:0"), temperature=0.0)
    with pytest.raises(TypeError):
        dg.linear_distill(x, w, t[:, None], torch.zeros(16, 1, device="cuda:0", dtype=torch.float64))
    with pytest.raises(ValueError):
        dg.linear_distill(x, w, t, torch.zeros(16, device="cuda:0"))
    with pytest.raises(TypeError):
        dg.linear_cross_entropy_backward(d["grad"].double(), x, w, t, lse)
    with pytest.raises(ValueError):
        dg.linear_cross_entropy_backward(d["grad"], x, w, t, lse, accumulate_dw=True)
    with pytest.raises(ValueError):
        dg.linear_cross_entropy_backward(d["grad"], x, w, t, lse, need_dx=False, dx=torch.empty_like(x))
    with pytest.raises(dg.GemmError):
        dg.linear_cross_entropy_backward(d["grad"], x, w, t, lse, dx=x)


# ---- masks and unusual values ---------------------------------------------------------------
@pytest.mark.parametrize("T", [1, 40, 300])
def test_no_row_has_a_target(dg, T):
    V, H = 500, 64
    d = on_gpu(make(T, V, H))
    d["target"].fill_(-100)
    loss, lse = call_forward(dg, d)
    dx, dw = call_backward(dg, d, lse)
    assert not loss.any() and not dx.any() and not dw.any()
    assert torch.isfinite(lse).all()
    e = on_gpu(make(T, V, H, K=5, kind="distill"))
    e["index"].fill_(-1)
    e["logits"].fill_(float("nan"))
    loss, lse = call_forward(dg, e)
    dx, dw = call_backward(dg, e, lse)
    assert not loss.any() and not dx.any() and not dw.any()


def test_another_ignore_index(dg):
    d = make(50, 300, 64, ignored=0.0)
    d["target"][::3] = 7
    g = on_gpu(d)
    f = oracle_forward(d, "bf16", ignore=7)
    loss, lse = call_forward(dg, g, ignore=7)
    dx, dw = call_backward(dg, g, lse, ignore=7)
    rx, rw, bx, bw = ol.backward(f, f64(d["x"]), f64(d["w"]), "bf16", f64(d["grad"]))
    assert ratio(f64(loss), f.loss, f.loss_bound) <= 1
    assert ratio(f64(dx), rx, bx) <= 1 and ratio(f64(dw), rw, bw) <= 1


@pytest.mark.parametrize("T", [6, 300])
def test_targets_out_of_range_are_loud(dg, T):
    V = 300
    d = on_gpu(make(T, V, 64, ignored=0.0))
    for i, bad in enumerate([V, V + 1000, -1, -101, 1 << 40]):
        d["target"][i] = bad
    loss, lse = call_forward(dg, d)
    assert torch.isnan(loss[:5]).all() and torch.isfinite(loss[5:]).all() and torch.isfinite(lse).all()
    dx, dw = call_backward(dg, d, lse)
    assert torch.isnan(dx[:5]).any(1).all() and torch.isfinite(dx[5:]).all()
    assert torch.isnan(dw).any()
    e = on_gpu(make(T, V, 64, K=4, kind="distill", ignored=0.0))
    e["index"][0, 2] = V
    e["index"][1, 0] = 1 << 33
    loss, lse = call_forward(dg, e)
    assert torch.isnan(loss[:2]).all() and torch.isfinite(loss[2:]).all()
    dx, dw = call_backward(dg, e, lse)
    assert torch.isnan(dx[:2]).any(1).all() and torch.isfinite(dx[2:]).all()


def check_distill(dg, d, dtype="bf16", tau=1.0, layout="nk"):
    f = oracle_forward(d, dtype, tau)
    g = on_gpu(d)
    loss, lse = call_forward(dg, g, layout, tau)
    dx, dw = call_backward(dg, g, lse, layout, tau)
    torch.cuda.synchronize()
    rx, rw, bx, bw = ol.backward(f, f64(d["x"]), f64(d["w"]), dtype, f64(d["grad"]), tau, distill=True)
    assert ratio(f64(loss), f.loss, f.loss_bound) <= 1
    assert ratio(f64(lse), f.lse, f.lse_bound) <= 1
    assert ratio(f64(dx), rx, bx) <= 1
    assert ratio(f64(dw) if layout == "nk" else f64(dw).T, rw, bw) <= 1
    return f, loss


@pytest.mark.parametrize("T", [7, 200])
def test_teacher_entries_that_are_masked_or_extreme(dg, T):
    d = make(T, 700, 64, K=6, kind="distill", ignored=0.0)
    inf = float("inf")
    d["logits"][0] = torch.tensor([1.0, -inf, 2.0, -inf, 0.5, 0.0])          # masked by -infinity
    d["logits"][1] = -inf                                                      # nothing left: no target
    d["logits"][2] = torch.finfo(torch.float32).min                            # the lowest value: a uniform row
    d["index"][3, 1:] = -1                                                     # one entry
    d["logits"][3, 1:] = float("nan")                                          # whatever padding holds
    d["index"][4, ::2] = -7
    d["logits"][4, ::2] = inf
    d["logits"][5] = torch.tensor([80.0, 0.0, -80.0, -500.0, 3.0, 1.0])        # entries whose weight vanishes
    f, loss = check_distill(dg, d)
    assert not f.on[1] and loss[1].item() == 0.0 and f.on[2]


def test_the_same_entry_twice(dg):
    d = make(60, 400, 64, K=8, kind="distill", ignored=0.0)
    d["index"][:, 3] = d["index"][:, 0]
    d["index"][:, 7] = d["index"][:, 0]
    d["index"][:30] = 5
    check_distill(dg, d, tau=2.0)


@pytest.mark.parametrize("K", [1, 63, 64, 65, 200, 1024])
def test_numbers_of_entries(dg, K):
    d = make(37, 1500, 72, K=K, kind="distill", seed=K)
    check_distill(dg, d, tau=1.5)
    # crowded into few tiles, the first and the last entries among them
    d["index"] = torch.where(d["index"] >= 0, d["index"] % 90 + torch.where(d["index"] % 2 == 0, 0, 1410), -1)
    check_distill(dg, d, tau=1.5)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_teacher_logits_in_16_bits(dg, dtype):
    d = make(70, 600, 64, K=9, kind="distill")
    d["logits"] = d["logits"].to(dtype)
    check_distill(dg, d, tau=2.0)


def test_logits_of_minus_infinity_and_large_ones(dg):
    # entries that a row of w holds at -infinity take no part; a target among them costs infinity
    T, V, H = 40, 300, 64
    d = make(T, V, H, ignored=0.0)
    d["x"] = d["x"].abs() + 0.125
    d["w"][5] = -float("inf")
    d["target"][:] = torch.where(d["target"] == 5, 6, d["target"])
    d["target"][0] = 5
    f = oracle_forward(d, "bf16")
    loss, lse = call_forward(dg, on_gpu(d))
    assert loss[0].item() == float("inf")
    g = dict(d, w=d["w"].clone())
    g["w"][5] = 0.0
    keep = oracle_forward(g, "bf16")   # for the bounds, which infinity would spoil
    z = f64(d["x"]) @ f64(d["w"]).T
    want = np.log(np.exp(z - np.where(np.isfinite(z), z, -np.inf).max(1, keepdims=True)).sum(1)) + z.max(1)
    assert ratio(f64(lse), want, keep.lse_bound) <= 1
    # logits in the hundreds: the statistics subtract the maximum
    d = make(T, V, H, spread=200.0)
    f = oracle_forward(d, "bf16")
    loss, lse = call_forward(dg, on_gpu(d))
    assert f.lse.max() > 300
    assert ratio(f64(loss), f.loss, f.loss_bound) <= 1 and ratio(f64(lse), f.lse, f.lse_bound) <= 1


def test_an_ignored_rows_infinite_logits_stay_its_own(dg):
    d = on_gpu(make(200, 300, 64, "fp16", ignored=0.0))
    clean_loss, clean_lse = call_forward(dg, d)
    d["target"][3] = -100
    clean = call_backward(dg, d, clean_lse)
    lse = clean_lse.clone()
    lse[3] = float("nan")
    dx, dw = call_backward(dg, d, lse)
    assert torch.equal(dx, clean[0]) and torch.equal(dw, clean[1])


@pytest.mark.parametrize("scale", [1e-30, 1e-6, 1.0, 1e4, 1e20])
def test_fp16_gradients_of_any_size(dg, scale):
    # the row factors' size is divided out of dz: what reaches fp16 does not depend on it
    T, V, H = 130, 900, 64
    d = make(T, V, H, "fp16", seed=9)
    d["grad"] = (d["grad"].abs() + 0.5) * scale
    g = on_gpu(d)
    loss, lse = call_forward(dg, g)
    dw = torch.empty(V, H, dtype=torch.float32, device="cuda:0")
    call_backward(dg, g, lse, need_dx=False, dw=dw)
    f = oracle_forward(d, "fp16")
    _, rw, _, bw = ol.backward(f, f64(d["x"]), f64(d["w"]), "fp16", f64(d["grad"]), dw_type="fp32")
    assert ratio(f64(dw), rw, bw) <= 1


def test_no_rows(dg):
    x = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda:0")
    w = torch.ones(100, 64, dtype=torch.bfloat16, device="cuda:0")
    t = torch.empty(0, dtype=torch.int64, device="cuda:0")
    loss, lse = dg.linear_cross_entropy(x, w, t)
    assert loss.shape == lse.shape == (0,)
    dx, dw = dg.linear_cross_entropy_backward(loss, x, w, t, lse)
    assert dx.shape == (0, 64) and dw.shape == w.shape and not dw.any()
    full, view = guarded(100, 64, 80, torch.float32)
    dg.linear_cross_entropy_backward(loss, x, w, t, lse, dw=view)
    assert not view.any() and guards_hold(full, view, 80)
    acc = torch.ones(100, 64, device="cuda:0")
    dg.linear_cross_entropy_backward(loss, x, w, t, lse, dw=acc, accumulate_dw=True)
    assert torch.equal(acc, torch.ones_like(acc))


# ---- runs, streams, graphs, workspaces --------------------------------------------------------
@pytest.mark.parametrize("shape", [(3, 5000, 264, "nk"), (60, 5000, 264, "kn"), (300, 5000, 264, "nk"), (1500, 5000, 264, "kn")], ids=str)
def test_every_run_gives_the_same_bits(dg, shape):
    T, V, H, layout = shape
    g = on_gpu(make(T, V, H, K=30, kind="distill", seed=11))
    loss, lse = call_forward(dg, g, layout, 2.0)
    dx, dw = call_backward(dg, g, lse, layout, 2.0)
    for _ in range(5):
        l2, e2 = call_forward(dg, g, layout, 2.0)
        x2, w2 = call_backward(dg, g, lse, layout, 2.0)
        assert torch.equal(loss, l2) and torch.equal(lse, e2) and torch.equal(dx, x2) and torch.equal(dw, w2)


@pytest.mark.parametrize("shape", [(3, 5000, 264, "nk"), (60, 5000, 264, "kn"), (300, 5000, 264, "nk"), (1500, 5000, 264, "kn")], ids=str)
def test_whatever_the_workspace_holds(dg, shape):
    T, V, H, layout = shape
    g = on_gpu(make(T, V, H, "fp16", K=30, kind="distill", seed=12))
    loss, lse = call_forward(dg, g, layout)
    dx, dw = call_backward(dg, g, lse, layout)
    for byte in (0, 0xFF):
        ws = torch.full((256 << 20,), byte, dtype=torch.uint8, device="cuda:0")
        l2, e2 = call_forward(dg, g, layout, workspace=ws)
        ws.fill_(byte)
        x2, w2 = call_backward(dg, g, lse, layout, workspace=ws)
        assert torch.equal(loss, l2) and torch.equal(lse, e2) and torch.equal(dx, x2) and torch.equal(dw, w2)


def test_two_streams_at_once(dg):
    jobs = [on_gpu(make(700, 9000, 264, seed=13)), on_gpu(make(40, 9000, 264, K=12, kind="distill", seed=14))]
    want = []
    for g in jobs:
        loss, lse = call_forward(dg, g)
        want.append((loss, lse) + call_backward(dg, g, lse))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    got = [None, None]
    for _ in range(6):
        for k, (g, s) in enumerate(zip(jobs, streams)):
            loss, lse = call_forward(dg, g, stream=s)
            got[k] = (loss, lse) + call_backward(dg, g, lse, stream=s)
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("kind", [("xent", 0), ("distill", 10)], ids=lambda k: k[0])
@pytest.mark.parametrize("T", [5, 300])
def test_captured_and_replayed(dg, T, kind):
    V, H = 3000, 136
    name, K = kind
    g = on_gpu(make(T, V, H, "fp16", K=K, kind=name, seed=15))
    call_forward(dg, g)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    say(f"  capture {name} T={T}")
    with torch.cuda.graph(graph):
        loss, lse = call_forward(dg, g)
        dx, dw = call_backward(dg, g, lse)
    for r in range(4):
        for k, v in on_gpu(make(T, V, H, "fp16", K=K, kind=name, seed=20 + r)).items():
            g[k].copy_(v)
        for t in (loss, lse, dx, dw):
            t.fill_(7.0)
        say(f"  replay {r}")
        graph.replay()
        torch.cuda.synchronize()
        l2, e2 = call_forward(dg, g)   # eager work between the replays
        x2, w2 = call_backward(dg, g, e2)
        torch.cuda.synchronize()
        assert torch.equal(loss, l2) and torch.equal(lse, e2) and torch.equal(dx, x2) and torch.equal(dw, w2)
    del graph


def raw_args(dg, g, loss, lse, dx=None, dw=None):
    T, H = g["x"].shape
    a = dg.GemmLossArgs(T=T, V=g["w"].shape[0], H=H, layout=dg.layout_word("nk", "bf16"), ignore_index=-100,
                        x=g["x"].data_ptr(), w=g["w"].data_ptr(), target=g["target"].data_ptr(), loss=loss.data_ptr(),
                        lse=lse.data_ptr(), grad=g["grad"].data_ptr())
    if dx is not None:
        a.dx, a.dw = dx.data_ptr(), dw.data_ptr()
    a.stream = torch.cuda.current_stream().cuda_stream
    return a


@pytest.mark.filterwarnings("ignore:The CUDA Graph is empty")
def test_the_c_calls_on_the_library_workspace(dg):
    g = on_gpu(make(300, 2000, 136, seed=16))
    loss, lse = call_forward(dg, g)
    dx, dw = call_backward(dg, g, lse)
    out = [torch.full_like(t, 7.0) for t in (loss, lse, dx, dw)]
    torch.cuda.synchronize()
    dg.gemm_release()
    graph, status = torch.cuda.CUDAGraph(), None
    with torch.cuda.graph(graph):   # nothing is there yet and nothing may be allocated now
        status = dg.gemm_loss_forward(raw_args(dg, g, *out))
    assert status == dg.GEMM_ERR_WORKSPACE
    del graph
    torch.cuda.synchronize()
    assert torch.all(out[0] == 7.0)
    assert dg.gemm_loss_forward(raw_args(dg, g, *out)) == dg.GEMM_OK, dg.gemm_last_error()
    assert dg.gemm_loss_backward(raw_args(dg, g, *out)) == dg.GEMM_OK, dg.gemm_last_error()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, (loss, lse, dx, dw)))
    # products on the same workspace before and after
    a, b = g["x"], g["w"].t().contiguous()
    c = torch.empty(300, 2000, device="cuda:0")
    dg.gemm_tensors(a, b, c, mode="streamk", splits=100)
    assert dg.gemm_loss_forward(raw_args(dg, g, *out)) == dg.GEMM_OK
    dg.gemm_tensors(a, b, c, mode="streamk", splits=100)
    assert dg.gemm_sync_status() == 0
    assert torch.equal(out[0], loss)
    want = f64(a) @ f64(g["w"]).T
    assert np.abs(f64(c) - want).max() <= 1e-4 * (np.abs(f64(a)) @ np.abs(f64(g["w"]).T)).max()


def test_offsets_beyond_32_bits(dg):
    # w of 4.3 GB: rows behind 2^31 elements and 2^32 bytes
    T, V, H = 4, 600000, 4096
    assert V * H > 1 << 31
    torch.manual_seed(3)
    x = torch.randn(T, H, device="cuda:0").bfloat16()
    w = torch.empty(V, H, dtype=torch.bfloat16, device="cuda:0")
    w.normal_().mul_(2.0 / 64)
    target = torch.tensor([0, V // 2, V - 1, V - 129], device="cuda:0")
    say("  forward")
    loss, lse = dg.linear_cross_entropy(x, w, target)
    z = torch.cat([(x.double() @ w[i: i + 50000].double().t()) for i in range(0, V, 50000)], 1)
    want = torch.logsumexp(z, 1)
    bound = 2 * (H / 16 + 8) * ol.F32 * 400 + 400 * ol.F32   # sum |x||w| is below 400 here
    assert (x.abs().double().sum(1) * w.abs().max().double()).max() > 0
    assert float((lse.double() - want).abs().max()) <= 4 * bound
    assert float((loss.double() - (want - z[torch.arange(T), target])).abs().max()) <= 8 * bound
    say("  backward")
    grad = torch.ones(T, device="cuda:0")
    dx, dw = dg.linear_cross_entropy_backward(grad, x, w, target, lse)
    p = torch.exp(z - want[:, None])
    p[torch.arange(T), target] -= 1.0
    rows = torch.tensor([0, 1, V // 2, V - 130, V - 129, V - 2, V - 1], device="cuda:0")
    ref = p[:, rows].t() @ x.double()
    # dz and dw rounded to bf16 once each, half a step 2^-8 of a value, over four rows; and p's own error
    tol = 2.0 ** -8 * (p[:, rows].abs().t() @ x.double().abs() + ref.abs()) + 8 * bound * (p[:, rows].abs().t() @ x.double().abs())
    assert bool(((dw[rows].double() - ref).abs() <= tol).all())
    refx = sum(p[:, i: i + 50000] @ w[i: i + 50000].double() for i in range(0, V, 50000))
    size = sum(p[:, i: i + 50000].abs() @ w[i: i + 50000].double().abs() for i in range(0, V, 50000))
    assert bool(((dx.double() - refx).abs() <= (2.0 ** -8 + 8 * bound + 2 * (V / 16 + 72) * ol.F32) * size + 2.0 ** -8 * refx.abs()).all())


# ---- together, as a training step uses them ------------------------------------------------------
def test_a_distillation_step_with_both_losses(dg):
    # loss = mean cross entropy + 0.5 x mean divergence over one micro-batch of hidden
    # states; dx adds up, dw accumulates in fp32 over the two losses and two micro-batches
    T, V, H, tau, zeta = 400, 3000, 264, 2.0, 1e-3
    dw = torch.zeros(V, H, device="cuda:0")
    rw, bw = np.zeros((V, H)), np.zeros((V, H))
    w = None
    for step in range(2):
        d = make(T, V, H, "bf16", seed=30 + step)
        if w is not None:
            d["w"] = w
        w = d["w"]
        e = make(T, V, H, "bf16", seed=40 + step, K=16, kind="distill")
        e["x"], e["w"] = d["x"], d["w"]
        n = int((d["target"] != -100).sum())
        d["grad"] = torch.full((T,), 1.0 / n)
        e["grad"] = torch.full((T,), 0.5 / T)
        gd, ge = on_gpu(d), on_gpu(e)
        ce, lse = call_forward(dg, gd, zeta=zeta)
        kd, lse_tau = call_forward(dg, ge, tau=tau)
        total = ce.sum() / n + 0.5 * kd.mean()
        dx1, _ = call_backward(dg, gd, lse, zeta=zeta, dw=dw, accumulate_dw=True)
        dx2, _ = call_backward(dg, ge, lse_tau, tau=tau, dw=dw, accumulate_dw=True)
        dx = dx1.float() + dx2.float()
        torch.cuda.synchronize()
        fd, fe = oracle_forward(d, "bf16", zeta=zeta), oracle_forward(e, "bf16", tau)
        want = fd.loss.sum() / n + 0.5 * fe.loss.mean()
        slack = fd.loss_bound.sum() / n + 0.5 * fe.loss_bound.mean() + 64 * ol.F32 * abs(want)
        assert abs(total.item() - want) <= slack
        x64, w64 = f64(d["x"]), f64(d["w"])
        a = ol.backward(fd, x64, w64, "bf16", f64(d["grad"]), 1.0, zeta, dw_type="fp32")
        b = ol.backward(fe, x64, w64, "bf16", f64(e["grad"]), tau, distill=True, dw_type="fp32")
        assert ratio(f64(dx), a[0] + b[0], a[2] + b[2] + ol.F32 * (np.abs(a[0]) + np.abs(b[0]))) <= 1
        rw += a[1] + b[1]
        bw += a[3] + b[3] + 2 * ol.F32 * np.abs(rw)   # the running sum's roundings
    assert ratio(f64(dw), rw, bw) <= 1
