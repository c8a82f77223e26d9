"""The feed-forward block and the adapters on a GPU: strides and guards, result types,
rows that are left out or broken, streams, graphs, workspaces, far offsets, and a
run of them together with a vocabulary loss."""
import math

import pytest
import torch

import ffn_util as fu
import lora_util as lu

pytestmark = pytest.mark.gpu
DEV = "cuda"
FFN = ("dx", "dw_gate", "dw_up", "dw_down")


@pytest.fixture(scope="module")
def dg():
    import dense_gemm_work_amd as dg

    assert torch.cuda.is_available(), "GPU test run without a visible GPU"
    return dg


def bits(t):
    return t.view(torch.int16 if t.element_size() == 2 else torch.int32)


def same(a, b):
    return all(torch.equal(bits(x), bits(y)) for x, y in zip(a, b))


GUARD = 11.0


def strided(t, extra, value=None):
    """(buffer, view): t's values, or `value`, in a view of a wider buffer of GUARD; its rows start 16 bytes in."""
    rows, cols = t.shape
    unit = 16 // t.element_size()
    buf = torch.full((rows + 2, unit + cols + extra), GUARD, dtype=t.dtype, device=t.device)
    view = buf[1:rows + 1, unit:unit + cols]
    view.copy_(t if value is None else torch.full_like(t, value))
    return buf, view


def guards(buf, view):
    keep = view.clone()
    view.fill_(GUARD)
    ok = bool((buf == GUARD).all())
    view.copy_(keep)
    return ok


# ---- strides ------------------------------------------------------------------------------
@pytest.mark.parametrize("T", [3, 40, 200])
@pytest.mark.parametrize("layout", ["nk", "kn"])
def test_ffn_strides(dg, layout, T):
    d = fu.make(T, 136, 264, "bf16", seed=T, dev=DEV)
    ws = [fu.stored(d[w], layout) for w in fu.WEIGHTS]
    want = fu.call_forward(dg, d, layout, save=True)
    grads = fu.call_backward(dg, d, layout)
    views = [strided(t, 8 * (i + 1))[1] for i, t in enumerate((d["x"], *ws))]
    outs = [strided(t, 16, 7.0) for t in want]
    got = dg.gated_ffn(*views, b_layout=layout, y=outs[0][1], gate=outs[1][1], up=outs[2][1])
    assert same(got, want) and all(guards(*o) for o in outs)
    gate, up, dy = (strided(d[k], 24)[1] for k in ("gate", "up", "dy"))
    outs = [strided(t, 8, 7.0) for t in grads]
    got = dg.gated_ffn_backward(dy, *views, gate, up, b_layout=layout, **{n: o[1] for n, o in zip(FFN, outs)})
    # w_gate's and w_up's strides differ: dx comes from two products instead of one sum
    want_dx = fu.oracle_backward(d, "silu", "bf16")["dx"]
    assert fu.ratio(got[0], want_dx) <= 1
    assert same(got[1:], grads[1:]) and all(guards(*o) for o in outs)


@pytest.mark.parametrize("T", [3, 40, 100, 200])
@pytest.mark.parametrize("layout", ["nk", "kn"])
def test_lora_strides(dg, layout, T):
    d = lu.make(T, 136, 264, 3, 72 if T == 100 else 16, "fp16", seed=T, dev=DEV)
    w, a, b = (lu.stored(d[k], layout) for k in ("w", "a", "b"))
    want = lu.call_forward(dg, d, layout)
    grads = lu.call_backward(dg, d, layout)
    x, wv, dy = strided(d["x"], 8)[1], strided(w, 24)[1], strided(d["dy"], 16)[1]
    wide = torch.full((3, 2, *a.shape[1:]), float("nan"), dtype=a.dtype, device=DEV)   # adapters between others
    wide[:, 0] = a
    av = wide[:, 0]
    bv = torch.cat((b.flatten(1), torch.full_like(b.flatten(1)[:, :8], float("nan"))), 1)[:, :-8].view_as(b) if T == 3 else b
    y = strided(want, 8, 7.0)
    assert same([dg.linear_lora(x, wv, av, bv, d["adapter"], scale=d["scale"], b_layout=layout, y=y[1])], [want]) and guards(*y)
    dx = strided(grads[0], 40, 7.0)
    got = dg.linear_lora_backward(dy, x, wv, av, bv, d["adapter"], scale=d["scale"], b_layout=layout, dx=dx[1])
    assert same(got, grads) and guards(*dx)


# ---- result types, parts of results -----------------------------------------------------------
@pytest.mark.parametrize("T", [20, 300, 3000])
@pytest.mark.parametrize("layout", ["nk", "kn"])
def test_fp32_gradients_and_sums(dg, layout, T):
    d = fu.make(T, 136, 200, "bf16", seed=T, dev=DEV)
    want = fu.oracle_backward(d, "gelu", "bf16", dw_type="fp32")
    new = [torch.full(tuple(fu.stored(d[w], layout).shape), 7.0, device=DEV) for w in fu.WEIGHTS]
    got = fu.call_backward(dg, d, layout, "gelu", **dict(zip(FFN[1:], new)))
    for name, t in zip(FFN[1:], got[1:]):
        assert t.dtype == torch.float32 and fu.ratio(fu.stored(t, layout), want[name]) <= 1, name
    total = [torch.randn_like(t) for t in new]
    before = [t.clone() for t in total]
    fu.call_backward(dg, d, layout, "gelu", accumulate_dw=True, **dict(zip(FFN[1:], total)))
    assert all(torch.equal(t, b + n) for t, b, n in zip(total, before, new))   # one fp32 addition
    e = lu.make(T, 136, 200, 5, 16, "bf16", seed=T, dev=DEV)
    want = lu.oracle_backward(e, "bf16", dab_type="fp32")
    new = [torch.full(tuple(lu.stored(e[k], layout).shape), 7.0, device=DEV) for k in ("a", "b")]
    got = lu.call_backward(dg, e, layout, da=new[0], db=new[1])
    for name, t in zip(("da", "db"), got[1:]):
        assert lu.ratio(lu.stored(t, layout), want[name]) <= 1, name
    total = [torch.randn_like(t) for t in new]
    before = [t.clone() for t in total]
    lu.call_backward(dg, e, layout, da=total[0], db=total[1], accumulate_dab=True)
    assert all(torch.equal(t, b + n) for t, b, n in zip(total, before, new))


@pytest.mark.parametrize("T", [20, 300])
def test_results_that_are_not_asked_for(dg, T):
    d, e = fu.make(T, 136, 200, seed=1, dev=DEV), lu.make(T, 136, 200, 5, 16, seed=1, dev=DEV)
    full, low = fu.call_backward(dg, d), lu.call_backward(dg, e)
    only = fu.call_backward(dg, d, need_dw=False)
    assert only[1:] == (None,) * 3 and same(only[:1], full[:1])
    only = fu.call_backward(dg, d, need_dx=False)
    assert only[0] is None and same(only[1:], full[1:])
    only = lu.call_backward(dg, e, need_dab=False)
    assert only[1:] == (None, None) and same(only[:1], low[:1])
    only = lu.call_backward(dg, e, need_dx=False)
    assert only[0] is None and same(only[1:], low[1:])
    # single ones by the C calls
    for keep in FFN[1:]:
        a = dg.ffn._block(d["x"], *(d[w] for w in fu.WEIGHTS), "silu", "nk")
        a.dy = d["dy"].data_ptr()
        dg.ffn._hidden(a, d["x"], d["gate"], d["up"])
        t = torch.empty_like(full[FFN.index(keep)])
        setattr(a, keep, t.data_ptr())
        dg.ffn._call(a, d["x"], True, None)
        assert same([t], [full[FFN.index(keep)]])
    for i, keep in ((1, "da"), (2, "db")):
        p = dg.lora._projection(e["x"], e["w"], e["a"], e["b"], e["adapter"], e["scale"], "nk")
        p.dy = e["dy"].data_ptr()
        t = torch.empty_like(low[i])
        setattr(p, keep, t.data_ptr())
        dg.lora._call(p, e["x"], True, None)
        assert same([t], [low[i]])


def test_no_rows(dg):
    d, e = fu.make(0, 64, 96, dev=DEV), lu.make(0, 64, 96, 2, 8, order="none", dev=DEV)
    y, gate, up = fu.call_forward(dg, d, save=True)
    assert y.shape == (0, 64) and gate.shape == up.shape == (0, 96)
    got = fu.call_backward(dg, d)
    assert got[0].shape == (0, 64) and all(int(torch.count_nonzero(t)) == 0 for t in got[1:])
    assert lu.call_forward(dg, e).shape == (0, 96)
    got = lu.call_backward(dg, e)
    assert got[0].shape == (0, 64) and all(int(torch.count_nonzero(t)) == 0 for t in got[1:])
    total = torch.ones(2, 8, 64, device=DEV), torch.ones(2, 96, 8, device=DEV)
    lu.call_backward(dg, e, da=total[0], db=total[1], accumulate_dab=True)
    assert all(bool((t == 1).all()) for t in total)


# ---- rows and adapters that are left out, out of range or broken ----------------------------------
@pytest.mark.parametrize("T", [1, 4, 60, 100, 300])
@pytest.mark.parametrize("layout", ["nk", "kn"])
def test_rows_without_an_adapter_are_the_plain_product(dg, layout, T):
    d = lu.make(T, 264, 520, 3, 16, "bf16", "none", seed=T, dev=DEV)
    w, a, b = (lu.stored(d[k], layout) for k in ("w", "a", "b"))
    nan = torch.full_like(a, float("nan")), torch.full_like(b, float("inf"))   # nothing of them is read
    y = dg.linear_lora(d["x"], w, *nan, d["adapter"], b_layout=layout)
    assert lu.ratio(y, lu.oracle_forward(d, "bf16")) <= 1
    dx, da, db = dg.linear_lora_backward(d["dy"], d["x"], w, *nan, d["adapter"], b_layout=layout)
    assert lu.ratio(dx, lu.oracle_backward(d, "bf16")["dx"]) <= 1
    assert int(torch.count_nonzero(da)) == 0 and int(torch.count_nonzero(db)) == 0


@pytest.mark.parametrize("shape", [(3, 16), (60, 16), (100, 16), (100, 64), (300, 16)], ids=str)
def test_adapters_out_of_range(dg, shape):
    T, R = shape
    d = lu.make(T, 264, 520, 3, R, "bf16", seed=T, dev=DEV)
    d["adapter"][1] = 3
    d["adapter"][T - 1] = 2 ** 40
    assert lu.ratio(lu.call_forward(dg, d), lu.oracle_forward(d, "bf16")) <= 1
    got, want = lu.call_backward(dg, d), lu.oracle_backward(d, "bf16")
    assert all(lu.ratio(t, want[k]) <= 1 for k, t in zip(("dx", "da", "db"), got))
    assert bool(got[0][1].isnan().all()) and not bool(got[0][0].isnan().any())


@pytest.mark.parametrize("shape", [(4, 16), (60, 16), (100, 64), (300, 16)], ids=str)
def test_what_a_row_holds_stays_in_it(dg, shape):
    T, R = shape
    d = lu.make(T, 264, 520, 3, R, "bf16", seed=T, dev=DEV)
    d["adapter"][: T // 2] = torch.arange(T // 2, device=DEV) % 2        # adapter 2 has no row of these
    d["adapter"][T // 2:] = 2
    y, grads = lu.call_forward(dg, d), lu.call_backward(dg, d)
    for value in (float("nan"), float("inf")):
        e = dict(d, x=d["x"].clone(), dy=d["dy"].clone())
        e["x"][T - 1], e["dy"][T - 1] = value, value
        assert same([lu.call_forward(dg, e)[:-1]], [y[:-1]])
        dx, da, db = lu.call_backward(dg, e)
        assert same([dx[:-1], da[:2], db[:2]], [grads[0][:-1], grads[1][:2], grads[2][:2]])
        assert bool(dx[-1].isnan().any()) and bool(da[2].isnan().any())
    f = fu.make(T, 136, 200, seed=T, dev=DEV)
    y = fu.call_forward(dg, f)
    f["x"][T - 1] = float("nan")
    assert same([fu.call_forward(dg, f)[:-1]], [y[:-1]])


def test_scale_may_be_left_out(dg):
    d = lu.make(70, 136, 200, 3, 16, seed=1, dev=DEV)
    d["scale"] = torch.ones(3, device=DEV)
    want = [lu.call_forward(dg, d), *lu.call_backward(dg, d)]
    args = (d["x"], d["w"], d["a"], d["b"], d["adapter"])
    assert same([dg.linear_lora(*args), *dg.linear_lora_backward(d["dy"], *args)], want)


def test_large_gates(dg):
    # silu and gelu far out, where their exponentials leave fp32's range
    d = fu.make(70, 64, 64, "bf16", seed=1, dev=DEV)
    d["gate"] = torch.linspace(-300, 300, 70 * 64, device=DEV).to(torch.bfloat16).view(70, 64)
    for act in ("silu", "gelu", "relu"):
        got, want = fu.call_backward(dg, d, act=act), fu.oracle_backward(d, act, "bf16")
        assert all(fu.ratio(t, want[k]) <= 1 for k, t in zip(FFN, got)), act
    d["x"] = (d["x"].float() * 60).to(torch.bfloat16)
    for act in ("silu", "gelu", "relu"):
        got, want = fu.call_forward(dg, d, act=act, save=True), fu.oracle_forward(d, act, "bf16")
        assert all(fu.ratio(t, want[k]) <= 1 for k, t in zip(("y", "gate", "up"), got)), act


@pytest.mark.parametrize("layout", ["nk", "kn"])
@pytest.mark.parametrize("T", [2, 5, 40, 65, 700])
def test_hidden_values_beyond_fp16(dg, layout, T):
    # h, dg and du overflow to infinities and every weight is positive: y and dx are infinite, not NaN (h stays
    # fp32 up to 4 rows of "nk": 128 features of 256 * 512 / 2^14 each are 1024 there, exactly)
    H, F = 64, 128
    one = lambda *s: torch.ones(*s, dtype=torch.float16, device=DEV)
    x, wg, wu, wd = one(T, H), one(F, H) * 4, one(F, H) * 8, one(H, F) * 2.0 ** -14
    stored = [fu.stored(w, layout) for w in (wg, wu, wd)]
    y, gate, up = dg.gated_ffn(x, *stored, activation="relu", b_layout=layout, save=True)
    assert bool((gate == 256).all()) and bool((up == 512).all())
    whole = layout == "nk" and T <= 4
    assert bool((y == (1024 if whole else math.inf)).all())
    dy = one(T, H) * 2.0 ** 13                                    # dh = 2^13 * 64 / 2^14 = 32; dg, du = 2^14, 2^13: in range
    dx, _, _, _ = dg.gated_ffn_backward(dy, x, *stored, gate, up, activation="relu", b_layout=layout)
    assert bool((dx == math.inf).all())                           # 128 * (2^14 * 4 + 2^13 * 8) in fp16
    dx, dwg, dwu, dwd = dg.gated_ffn_backward(dy * 4, x, *stored, gate, up * 2, activation="relu", b_layout=layout)
    assert all(bool((t == math.inf).all()) for t in (dx, dwg, dwd))   # dg = 2^17, h = 2^18; du = 2^15 is in range
    assert not bool(dwu.isnan().any())


@pytest.mark.parametrize("act", ["silu", "gelu", "relu"])
@pytest.mark.parametrize("T", [3, 40, 200])
def test_nan_gates_stay_nan(dg, act, T):
    d = fu.make(T, 64, 64, "bf16", seed=1, dev=DEV)
    d["w_gate"][5] = float("nan")
    d["w_down"][:, 5] = 1.0
    assert bool(fu.call_forward(dg, d, act=act).isnan().all())


# ---- streams, graphs, workspaces ---------------------------------------------------------------------
def everything(dg, d, e, **kw):
    return [*fu.call_forward(dg, d, save=True, **kw), *fu.call_backward(dg, d, **kw), lu.call_forward(dg, e, **kw),
            *lu.call_backward(dg, e, **kw)]


@pytest.mark.parametrize("T", [1, 30, 100, 700])
def test_the_same_call_gives_the_same_bits_on_any_stream(dg, T):
    d, e = fu.make(T, 264, 520, seed=T, dev=DEV), lu.make(T, 264, 520, 6, 16, seed=T, dev=DEV)
    want = everything(dg, d, e)
    torch.cuda.synchronize()
    side = [torch.cuda.Stream() for _ in range(2)]
    got = [everything(dg, d, e, stream=s) for s in side for _ in range(2)]
    torch.cuda.synchronize()
    assert all(same(g, want) for g in got)
    # a caller's workspace and the library's
    a = dg.ffn._block(d["x"], *(d[w] for w in fu.WEIGHTS), "silu", "nk")
    y = torch.empty_like(want[0])
    a.y = y.data_ptr()
    need = dg.gemm_ffn_plan(a, False, torch.cuda.get_device_properties(0).multi_processor_count).workspace_bytes
    ws = torch.full((need + 256,), 255, dtype=torch.uint8, device=DEV)
    assert same([fu.call_forward(dg, d, workspace=ws[:need])], want[:1]) and bool((ws[need:] == 255).all())
    a.stream = dg.current_stream_word(0)
    assert dg.gemm_ffn_forward(a) == dg.GEMM_OK
    torch.cuda.synchronize()
    assert same([y], want[:1])


@pytest.mark.parametrize("T", [1, 30, 100, 700])
def test_captured_and_replayed(dg, T):
    d, e = fu.make(T, 264, 520, seed=T, dev=DEV), lu.make(T, 264, 520, 6, 16, seed=T, dev=DEV)
    everything(dg, d, e)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = everything(dg, d, e)
    for i in range(4):   # new inputs, also new adapters, in the same memory
        for to, new in ((d, fu.make(T, 264, 520, seed=50 + i, dev=DEV)), (e, lu.make(T, 264, 520, 6, 16, seed=60 + i, dev=DEV))):
            for k in to:
                to[k].copy_(new[k])
        want = everything(dg, d, e)
        for t in got:
            t.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        assert same(got, want), i


def test_two_graphs_share_nothing(dg):
    d, e = fu.make(100, 264, 520, seed=1, dev=DEV), lu.make(100, 264, 520, 6, 64, seed=1, dev=DEV)
    want = everything(dg, d, e)
    graphs, got = [], []
    for _ in range(2):
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            got.append(everything(dg, d, e))
        graphs.append((g, side))
    for _ in range(3):
        for g, side in graphs:
            with torch.cuda.stream(side):
                g.replay()
        torch.cuda.synchronize()
        assert all(same(g, want) for g in got)


# ---- far offsets ------------------------------------------------------------------------------------
def test_offsets_beyond_32_bits(dg):
    T, far = 1100, 1 << 21                       # rows 4 MiB apart: the last at 4.6 GB
    d = fu.make(T, 64, 72, seed=1, dev=DEV)
    want = [*fu.call_forward(dg, d, save=True), *fu.call_backward(dg, d)]
    buf = torch.empty(T, far, dtype=torch.bfloat16, device=DEV)
    x, dy, gate, up, y, dx = (buf[:, 128 * i:128 * i + n] for i, n in enumerate((64, 64, 72, 72, 64, 64)))
    for to, k in ((x, "x"), (dy, "dy")):
        to.copy_(d[k])
    ws = [d[w] for w in fu.WEIGHTS]
    got = [t.clone() for t in dg.gated_ffn(x, *ws, y=y, gate=gate, up=up)]
    gate.copy_(d["gate"]), up.copy_(d["up"])
    assert same(got + list(dg.gated_ffn_backward(dy, x, *ws, gate, up, dx=dx)), want)
    e = lu.make(T, 64, 72, 3, 8, seed=1, dev=DEV)
    want = [lu.call_forward(dg, e), *lu.call_backward(dg, e)]
    x.copy_(e["x"])
    dy, y = buf[:, 1024:1096], buf[:, 1152:1224]
    dy.copy_(e["dy"])
    stride = 1 << 30                             # adapters 2 GiB apart
    store = torch.empty(2 * stride + 2048, dtype=torch.bfloat16, device=DEV)
    a, b = store.as_strided((3, 8, 64), (stride, 64, 1)), store.as_strided((3, 72, 8), (stride, 8, 1), 512)
    a.copy_(e["a"]), b.copy_(e["b"])
    args = (x, e["w"], a, b, e["adapter"])
    got = [dg.linear_lora(*args, scale=e["scale"], y=y).clone(), *dg.linear_lora_backward(dy, *args, scale=e["scale"], dx=dx)]
    assert same(got, want)


# ---- together ---------------------------------------------------------------------------------------
@pytest.mark.parametrize("T", [6, 90, 600])
def test_a_layer_and_a_loss_together(dg, T):
    """Adapters' projection, feed-forward block, vocabulary loss, forward and backward on the library's calls, against
    float64 autograd of the whole.  A chain of at most 8 values each rounded to bf16 (half a step, 2^-8, of each
    element) on the way forward and as many backward: relative error in the norm below 16 x 2^-8 where nothing
    amplifies it (the layers' weights keep the norms)."""
    H, F, V, R, L = 256, 520, 1000, 16, 4
    d, e = fu.make(T, H, F, seed=T, dev=DEV), lu.make(T, H, H, L, R, seed=T + 1, dev=DEV)
    g = torch.Generator(device=DEV).manual_seed(T)
    vocabulary = (torch.randn(V, H, device=DEV, generator=g) / math.sqrt(H)).to(torch.bfloat16)
    target = torch.randint(0, V, (T,), device=DEV, generator=g)
    grad = torch.full((T,), 1.0 / T, device=DEV)
    ws = [d[w] for w in fu.WEIGHTS]
    h = dg.linear_lora(e["x"], e["w"], e["a"], e["b"], e["adapter"], scale=e["scale"])
    y, gate, up = dg.gated_ffn(h, *ws, save=True)
    loss, lse = dg.linear_cross_entropy(y, vocabulary, target)
    dy, dv = dg.linear_cross_entropy_backward(grad, y, vocabulary, target, lse)
    dh, *dws = dg.gated_ffn_backward(dy, h, *ws, gate, up)
    dx, da, db = dg.linear_lora_backward(dh, e["x"], e["w"], e["a"], e["b"], e["adapter"], scale=e["scale"])
    leaves = [t.double().requires_grad_() for t in (e["x"], e["a"], e["b"], *ws, vocabulary)]
    x, a, b, wg, wu, wd, v = leaves
    i = e["adapter"].clamp(min=0)
    c = (e["scale"].double()[i] * (e["adapter"] >= 0))[:, None, None]
    h = x @ e["w"].double().t() + ((c * (x[:, None, :, None] * a[i].transpose(1, 2)[:, None]).sum(2)) [:, 0, :, None] * b[i].transpose(1, 2)).sum(1)
    out = (torch.nn.functional.silu(h @ wg.t()) * (h @ wu.t())) @ wd.t()
    total = torch.nn.functional.cross_entropy(out @ v.t(), target, reduction="none")
    (total / T).sum().backward()
    # a loss moves by at most twice what its row's logits move (lse by no more than the largest, its target's logit by
    # its own), a logit by no more than |dy| |v|, and |dy| is below 16 x 2^-8 |y| as above
    moves = 2 * 16 * 2.0 ** -8 * out.detach().norm(dim=1) * v.detach().norm(dim=1).max()
    assert bool(((loss.double() - total.detach()).abs() <= moves).all())
    for got, leaf in zip((dx, da, db, *dws, dv), leaves):
        rel = float((got.double() - leaf.grad).norm() / leaf.grad.norm())
        print(f"    {rel:.4f}", flush=True)
        assert rel < 16 * 2.0 ** -8
