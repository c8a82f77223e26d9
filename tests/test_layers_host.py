"""The feed-forward block and the adapters without a GPU: their 64-bit oracles against torch's
own functions and differences, the bounds' teeth, the planner, the torch-facing checks."""
import warnings

import pytest
import torch

from oracle import ffn as of
from oracle import lora as orc

import ffn_util as fu
import lora_util as lu


@pytest.fixture(scope="module")
def dg():
    import dense_gemm_work_amd as dg

    return dg


ACTS = {"silu": torch.nn.functional.silu, "gelu": torch.nn.functional.gelu, "relu": torch.relu}


@pytest.mark.parametrize("act", ACTS)
def test_ffn_oracle_is_torchs_definition(act):
    d = {k: v.double() for k, v in fu.make(7, 16, 24, seed=1).items()}
    leaves = {k: d[k].requires_grad_() for k in ("x", *fu.WEIGHTS)}
    x, wg, wu, wd = leaves.values()
    gate, up = x @ wg.t(), x @ wu.t()
    y = (ACTS[act](gate) * up) @ wd.t()
    f = of.forward(*(t.detach() for t in leaves.values()), act, "bf16")
    assert torch.allclose(f["y"][0], y.detach(), rtol=1e-12, atol=1e-13)
    y.backward(d["dy"])
    b = of.backward(d["dy"], *(t.detach() for t in leaves.values()), gate.detach(), up.detach(), act, "bf16")
    for name, leaf in zip(("dx", "dw_gate", "dw_up", "dw_down"), leaves.values()):
        assert torch.allclose(b[name][0], leaf.grad, rtol=1e-11, atol=1e-12), name


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_ffn_oracle_gradient_by_differences(act):
    d = {k: v.double() for k, v in fu.make(5, 8, 16, seed=2).items()}
    names = ("x", *fu.WEIGHTS)

    def total():
        return float((of.forward(*(d[n] for n in names), act, "bf16")["y"][0] * d["dy"]).sum())

    f = of.forward(*(d[n] for n in names), act, "bf16")
    b = of.backward(d["dy"], *(d[n] for n in names), f["gate"][0], f["up"][0], act, "bf16")
    for name, key in zip(names, ("dx", "dw_gate", "dw_up", "dw_down")):
        for at in [(0, 0), (2, 3), (4, 7)]:
            keep, h = float(d[name][at]), 1e-5
            d[name][at] = keep + h
            high = total()
            d[name][at] = keep - h
            low = total()
            d[name][at] = keep
            assert abs((high - low) / (2 * h) - float(b[key][0][at])) < 1e-7, (name, at)


def test_lora_oracle_is_torchs_definition_and_differences():
    d = lu.make(9, 16, 24, 3, 8, seed=3)
    d["adapter"][:3] = torch.tensor([-1, 0, 2])
    x, w, a, b = (d[k].double().requires_grad_() for k in ("x", "w", "a", "b"))
    dy, scale = d["dy"].double(), d["scale"].double()

    def forward(x, a, b):
        rows = [x[t] @ w.t() + (scale[i] * (x[t] @ a[i].t()) @ b[i].t() if i >= 0 else 0) for t, i in enumerate(d["adapter"].tolist())]
        return torch.stack(rows)

    y = forward(x, a, b)
    got, _ = orc.forward(x.detach(), w.detach(), a.detach(), b.detach(), d["adapter"], d["scale"], "bf16")
    assert torch.allclose(got, y.detach(), rtol=1e-12, atol=1e-13)
    y.backward(dy)
    g = orc.backward(dy, x.detach(), w.detach(), a.detach(), b.detach(), d["adapter"], d["scale"], "bf16")
    for name, leaf in (("dx", x), ("da", a), ("db", b)):
        assert torch.allclose(g[name][0], leaf.grad, rtol=1e-11, atol=1e-12), name
    with torch.no_grad():
        for leaf, name, at in ((x, "dx", (1, 5)), (a, "da", (2, 3, 4)), (b, "db", (0, 7, 1))):
            keep, h = float(leaf[at]), 1e-5
            leaf[at] = keep + h
            high = float((forward(x, a, b) * dy).sum())
            leaf[at] = keep - h
            low = float((forward(x, a, b) * dy).sum())
            leaf[at] = keep
            assert abs((high - low) / (2 * h) - float(g[name][0][at])) < 1e-7, name


def f32(d, dtype, *names):
    return [d[n].float() for n in names]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("act", ACTS)
def test_ffn_bounds_hold_for_an_fp32_evaluation_and_have_teeth(act, dtype):
    d = fu.make(120, 64, 200, dtype, seed=5)
    dt = fu.DTYPES[dtype]
    x, wg, wu, wd, dy, gate, up = f32(d, dtype, "x", *fu.WEIGHTS, "dy", "gate", "up")
    g, u = x @ wg.t(), x @ wu.t()
    h = (ACTS[act](g) * u).to(dt).float()
    want = fu.oracle_forward(d, act, dtype)
    for got, name in (((h @ wd.t()).to(dt), "y"), (g.to(dt), "gate"), (u.to(dt), "up")):
        assert fu.ratio(got, want[name]) <= 1, name
    assert fu.ratio((h @ wd.t()).to(dt), fu.oracle_forward(d, act, dtype, mutation=1)["y"]) > 1
    leaf = gate.clone().requires_grad_()
    slope, = torch.autograd.grad(ACTS[act](leaf).sum(), leaf)
    dh = dy @ wd
    dg, du = (dh * up * slope).to(dt).float(), (dh * ACTS[act](gate)).to(dt).float()
    h = (ACTS[act](gate) * up).to(dt).float()
    got = {"dx": dg @ wg + du @ wu, "dw_gate": dg.t() @ x, "dw_up": du.t() @ x, "dw_down": dy.t() @ h}
    want = fu.oracle_backward(d, act, dtype)
    for name, t in got.items():
        assert fu.ratio(t.to(dt), want[name]) <= 1, name
    assert fu.ratio(got["dw_gate"].to(dt), fu.oracle_backward(d, act, dtype, mutation=2)["dw_gate"]) > 1
    assert fu.ratio(got["dx"].to(dt), fu.oracle_backward(d, act, dtype, mutation=3)["dx"]) > 1


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_lora_bounds_hold_for_an_fp32_evaluation_and_have_teeth(dtype):
    d = lu.make(120, 64, 72, 4, 16, dtype, seed=6)
    dt = lu.DTYPES[dtype]
    x, w, a, b, dy = f32(d, dtype, "x", "w", "a", "b", "dy")
    on = d["adapter"] >= 0
    i = d["adapter"].clamp(min=0)
    c = (d["scale"][i] * on)[:, None]
    s = (c * (x[:, None] @ a[i].transpose(1, 2))[:, 0]).to(dt).float()
    y = x @ w.t() + (s[:, None] @ b[i].transpose(1, 2))[:, 0]
    assert lu.ratio(y.to(dt), lu.oracle_forward(d, dtype)) <= 1
    for m in (1, 2):
        assert lu.ratio(y.to(dt), lu.oracle_forward(d, dtype, mutation=m)) > 1
    ds = (c * (dy[:, None] @ b[i])[:, 0]).to(dt).float()
    dx = dy @ w + (ds[:, None] @ a[i])[:, 0]
    own = torch.nn.functional.one_hot(i, 4).float() * on[:, None]
    da, db = torch.einsum("tl,tr,th->lrh", own, ds, x), torch.einsum("tl,tn,tr->lnr", own, dy, s)
    want = lu.oracle_backward(d, dtype)
    for name, t in (("dx", dx), ("da", da), ("db", db)):
        assert lu.ratio(t.to(dt), want[name]) <= 1, name
    assert lu.ratio(da.to(dt), lu.oracle_backward(d, dtype, mutation=3)["da"]) > 1


def test_plans(dg):
    word = dg.layout_word("nk", "bf16")
    kn = dg.layout_word("kn", "bf16")

    def ffn(T, H, F, backward=False, layout=word):
        return dg.gemm_ffn_plan(dg.GemmFfnArgs(T=T, H=H, F=F, layout=layout, dx=1, dw_gate=1, dw_up=1, dw_down=1), backward, 256)

    assert ffn(4, 256, 512).parts == 0 and ffn(4, 256, 512, layout=kn).parts == 2     # h in fp32; in two parts
    assert ffn(64, 256, 512).parts == 2 and ffn(65, 256, 512).parts == 1
    assert ffn(4, 256, 512).workspace_bytes == 4 * 512 * 4
    p = ffn(8192, 4096, 12288)
    assert (p.first_tile_f, p.first_tile_t, p.out_splits, p.workspace_bytes) == (128, 256, 1, 8192 * 12288 * 2)
    p = ffn(8192, 4096, 12288, True)
    assert p.workspace_bytes == 3 * 8192 * 12288 * 2 and p.dw_splits == 1
    two = dg.gemm_ffn_plan(dg.GemmFfnArgs(T=8192, H=4096, F=12288, layout=word, dx=1, ldw_gate=4104), True, 256)
    assert two.workspace_bytes > p.workspace_bytes                                     # two strides: dx by way of slots

    def lora(T, H, N, R, L=4, backward=False):
        return dg.gemm_lora_plan(dg.GemmLoraArgs(T=T, H=H, N=N, R=R, adapters=L, layout=word, dx=1, da=1, db=1), backward, 256)

    for T, tile in ((1, 32), (32, 32), (33, 64), (64, 64), (65, 128), (128, 128)):
        assert lora(T, 1024, 1024, 16).out_tile_t == tile
    p = lora(5000, 4096, 8192, 64, 24)
    assert (p.out_tile_p, p.out_tile_t, p.out_whole, p.out_splits) == (256, 256, 512, 2)
    assert lora(8192, 4096, 4096, 64, 8).out_whole == 512
    for backward in (False, True):
        for T in (0, 1, 64, 65, 129, 5000, 70000):
            for R in (8, 64, 72, 1024):
                p = lora(T, 264, 1032, R, 3, backward)
                assert p.workspace_bytes >= 0 and p.out_splits >= 1 and p.low_splits >= 1 and p.low_lists >= 1


def test_tensor_checks(dg):
    d = fu.make(4, 16, 24)
    ws = [d[w] for w in fu.WEIGHTS]
    with pytest.raises(ValueError, match="device tensor"):
        dg.gated_ffn(d["x"], *ws)
    with pytest.raises(TypeError):
        dg.gated_ffn(d["x"].float(), *ws)
    with pytest.raises(ValueError, match="2-D"):
        dg.gated_ffn(d["x"][0], *ws)
    e = lu.make(4, 16, 24, 2, 8)
    with pytest.raises(ValueError, match="device tensor"):
        dg.linear_lora(e["x"], e["w"], e["a"], e["b"], e["adapter"])
    with pytest.raises(TypeError):
        dg.linear_lora(e["x"].float(), e["w"], e["a"], e["b"], e["adapter"])
    with pytest.raises(ValueError, match="3-D"):
        dg.linear_lora(e["x"], e["w"], e["a"][0], e["b"], e["adapter"])


def test_inputs_that_require_gradients_are_warned_about(dg):
    d, e = fu.make(4, 16, 24), lu.make(4, 16, 24, 2, 8)
    for n in ("x", *fu.WEIGHTS):
        g = dict(d, **{n: d[n].clone().requires_grad_()})
        with pytest.warns(UserWarning, match="not recorded for autograd"), pytest.raises(ValueError, match="device tensor"):
            dg.gated_ffn(g["x"], *(g[w] for w in fu.WEIGHTS))
    for n in ("x", "w", "a", "b"):
        g = dict(e, **{n: e[n].clone().requires_grad_()})
        with pytest.warns(UserWarning, match="not recorded for autograd"), pytest.raises(ValueError, match="device tensor"):
            dg.linear_lora(g["x"], g["w"], g["a"], g["b"], g["adapter"])
        with warnings.catch_warnings(), torch.no_grad():
            warnings.simplefilter("error")
            with pytest.raises(ValueError, match="device tensor"):
                dg.linear_lora(g["x"], g["w"], g["a"], g["b"], g["adapter"])
