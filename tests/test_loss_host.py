"""Vocabulary losses without a GPU: the fp64 oracle's pins, the planner, and the
calls that are refused before anything is launched."""
import ctypes
import subprocess
from pathlib import Path

import numpy as np
import pytest
import torch

from oracle import loss as ol

from loss_util import f64, make, oracle_forward, ratio

ROOT = Path(__file__).resolve().parent.parent


@pytest.fixture(scope="module")
def dg():
    import dense_gemm_work_amd as dg

    return dg


# ---- the oracle ---------------------------------------------------------------------
CASES = [("xent", 0, 1.0, 0.0), ("xent", 0, 1.0, 1e-2), ("distill", 5, 2.0, 0.0), ("distill", 3, 0.5, 0.0)]


def torch_loss(d, x, w, tau, zeta):
    """The losses by torch's own double-precision functions."""
    z = x @ w.t()
    if "target" in d:
        loss = torch.nn.functional.cross_entropy(z, d["target"], ignore_index=-100, reduction="none")
        return loss + torch.where(d["target"] == -100, 0.0, zeta * torch.logsumexp(z, 1) ** 2)
    s = torch.where(d["index"] >= 0, d["logits"].double() / tau, -torch.inf)
    q = torch.nan_to_num(torch.softmax(s, 1))
    log_p = torch.log_softmax(z / tau, 1).gather(1, d["index"].clamp(min=0))
    return tau * tau * (torch.special.xlogy(q, q) - q * log_p).sum(1)


@pytest.mark.parametrize("case", CASES, ids=str)
def test_oracle_is_torchs_definition(case):
    kind, K, tau, zeta = case
    d = make(40, 30, 16, kind=kind, K=K, seed=3)
    f = oracle_forward(d, "bf16", tau, zeta)
    x, w = d["x"].double().requires_grad_(), d["w"].double().requires_grad_()
    loss = torch_loss(d, x, w, tau, zeta)
    assert np.allclose(f.loss, loss.detach().numpy(), rtol=1e-12, atol=1e-12)
    loss.backward(d["grad"].double())
    dx, dw, _, _ = ol.backward(f, f64(d["x"]), f64(d["w"]), "bf16", f64(d["grad"]), tau, zeta, kind == "distill")
    assert np.allclose(dx, x.grad.numpy(), rtol=1e-11, atol=1e-12)
    assert np.allclose(dw, w.grad.numpy(), rtol=1e-11, atol=1e-12)


@pytest.mark.parametrize("case", CASES, ids=str)
def test_oracle_gradient_by_differences(case):
    kind, K, tau, zeta = case
    d = make(6, 11, 8, kind=kind, K=K, seed=4, ignored=0.0)
    g = f64(d["grad"])
    f = oracle_forward(d, "bf16", tau, zeta)
    dx, dw, _, _ = ol.backward(f, f64(d["x"]), f64(d["w"]), "bf16", g, tau, zeta, kind == "distill")

    def total(x, w):
        kw = dict(target=d["target"].numpy()) if kind == "xent" else dict(index=d["index"].numpy(), logits=f64(d["logits"]))
        return float((g * ol.forward(x, w, "bf16", tau=tau, zeta=zeta, **kw).loss).sum())

    x, w, h = f64(d["x"]), f64(d["w"]), 1e-5
    for arr, grad in ((x, dx), (w, dw)):
        for at in [(0, 0), (2, 3), (5, 7)]:
            keep = arr[at]
            arr[at] = keep + h
            up = total(x, w)
            arr[at] = keep - h
            down = total(x, w)
            arr[at] = keep
            assert abs((up - down) / (2 * h) - grad[at]) < 1e-6


def fp32_evaluation(d, tau, zeta):
    """A straightforward fp32 forward and backward on the CPU: loss, lse, dx, dw."""
    x, w = d["x"].float(), d["w"].float()
    z = x @ w.t() / tau
    lse = torch.logsumexp(z, 1)
    g = d["grad"]
    if "target" in d:
        on = d["target"] >= 0
        q = torch.zeros_like(z)
        q[on, d["target"][on]] = 1.0
        loss = torch.where(on, lse - (q * z).sum(1) + zeta * lse * lse, 0.0)
        a, b = g * (1 + 2 * zeta * lse), g
    else:
        s = torch.where(d["index"] >= 0, d["logits"] / tau, -torch.inf)
        qk = torch.nan_to_num(torch.softmax(s, 1))
        on = (d["index"] >= 0).any(1)
        q = torch.zeros(len(x), len(w) + 1).scatter_add_(1, torch.where(d["index"] < 0, len(w), d["index"]), qk)[:, :-1]
        loss = torch.where(on, tau * tau * (torch.special.xlogy(qk, qk).sum(1) - (q * z).sum(1) + lse), 0.0)
        a = b = g * tau
    dz = a[:, None] * torch.exp(z - lse[:, None]) - b[:, None] * q
    dz = torch.where(on[:, None], dz, 0.0).to(d["x"].dtype).float()
    return loss, lse, (dz @ w).to(d["x"].dtype), (dz.t() @ x).to(d["x"].dtype)


@pytest.mark.parametrize("dtype", ["bf16"])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_bounds_hold_for_an_fp32_evaluation_and_have_teeth(case, dtype):
    kind, K, tau, zeta = case
    d = make(120, 700, 64, dtype, kind=kind, K=K, seed=5)
    f = oracle_forward(d, dtype, tau, zeta)
    loss, lse, dx, dw = fp32_evaluation(d, tau, zeta)
    x, w, g = f64(d["x"]), f64(d["w"]), f64(d["grad"])
    rx, rw, bx, bw = ol.backward(f, x, w, dtype, g, tau, zeta, kind == "distill")
    assert ratio(f64(lse), f.lse, f.lse_bound) <= 1
    assert ratio(f64(loss), f.loss, f.loss_bound) <= 1
    assert ratio(f64(dx), rx, bx) <= 1 and ratio(f64(dw), rw, bw) <= 1
    # planted mistakes must fall outside
    if kind == "xent" and zeta:
        bad = ol.forward(x, w, dtype, target=d["target"].numpy(), zeta=zeta, mutation=1)
        assert ratio(f64(loss), bad.loss, bad.loss_bound) > 1
        mx, _, _, _ = ol.backward(f, x, w, dtype, g, tau, zeta, mutation=3)
        assert ratio(f64(dx), mx, bx) > 1
    if kind == "distill":
        bad = ol.forward(x, w, dtype, index=d["index"].numpy(), logits=f64(d["logits"]), tau=tau, mutation=2)
        assert ratio(f64(loss), bad.loss, bad.loss_bound) > 1
    mx, mw, _, _ = ol.backward(f, x, w, dtype, g, tau, zeta, kind == "distill", mutation=4)
    assert ratio(f64(dx), mx, bx) > 1 and ratio(f64(dw), mw, bw) > 1


# ---- the planner ----------------------------------------------------------------------
def args_of(dg, T=300, V=1000, H=128, layout=None, kind=0, entries=0, dx=1, dw=1, dw_type=0):
    a = dg.GemmLossArgs()
    a.T, a.V, a.H = T, V, H
    a.layout = dg.GEMM_B_NK if layout is None else layout
    a.kind, a.entries, a.dx, a.dw, a.dw_type = kind, entries, dx, dw, dw_type
    return a


def test_plans_cover_the_vocabulary_and_stay_small(dg):
    rng = np.random.default_rng(0)
    for _ in range(400):
        T, V, H = (int(np.exp(rng.uniform(0, np.log(m)))) for m in (1 << 20, 1 << 18, 1 << 10))
        V, H = max(V // 8 * 8, 8), 8 * max(H, 1)
        if T * V > dg.GEMM_LOSS_MAX_TV:
            continue
        layout = dg.GEMM_B_KN if rng.random() < 0.5 else dg.GEMM_B_NK
        kind = int(rng.random() < 0.3)
        entries = int(rng.integers(1, 200)) if kind else 0
        a = args_of(dg, T, V, H, layout, kind, entries, dx=int(rng.random() < 0.8), dw=int(rng.random() < 0.8))
        f = dg.gemm_loss_plan(a, False, 256)
        b = dg.gemm_loss_plan(a, True, 256)
        assert f.tile_v in (32, 64, 128, 256) and f.tile_t in (32, 64, 128, 256)
        assert f.workspace_bytes >= 12 * -(-V // f.tile_v) * T
        assert b.pieces == -(-V // b.piece) and b.piece % 64 == 0
        assert b.dx_splits >= 1 and b.dw_splits >= 1
        # dz of one piece: at most 256 MiB, or 1024 entries of the vocabulary
        assert T * b.piece * 2 <= 256 << 20 or b.piece <= 1024
        # the rest: dx's and dw's slices and what follows the teacher's entries
        slices = 4 * b.dx_splits * (T + 256) * (H + 256) + 4 * (b.dw_splits if b.dw_splits > 1 else 0) * (b.piece + 256) * (H + 256)
        assert b.workspace_bytes <= T * b.piece * 2 + slices + T * (entries * 8 + 256) + 8192


def test_few_rows_take_thin_tiles(dg):
    assert dg.gemm_loss_plan(args_of(dg, 1, 8192, 1536), False, 256).tile_v == 32
    p = dg.gemm_loss_plan(args_of(dg, 40, 50001, 2048), False, 256)
    assert (p.tile_v, p.tile_t) == (64, 64)
    p = dg.gemm_loss_plan(args_of(dg, 40, 50000, 2048, dg.GEMM_B_KN), True, 256)
    assert (p.tile_v, p.tile_t, p.dx_tile_h, p.dx_tile_t) == (128, 64, 128, 64)
    p = dg.gemm_loss_plan(args_of(dg, 8192, 131072, 4096), True, 256)
    assert (p.tile_v, p.tile_t, p.dx_tile_h, p.dw_tile_p) == (256, 256, 256, 256)


def test_header_compiles_as_c(tmp_path):
    src = tmp_path / "h.c"
    src.write_text('#include "gemm_loss.h"\nint main(void) { gemm_loss_args_t a = {0}; gemm_loss_plan_t p; '
                   'return (int)sizeof a + (int)sizeof p + a.entries == 0; }\n')
    subprocess.run(["gcc", "-std=c11", "-Wall", "-Werror", "-I", str(ROOT / "include"), "-c", str(src), "-o",
                    str(tmp_path / "h.o")], check=True)


def test_structures_match_the_header(dg, tmp_path):
    src = tmp_path / "s.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "gemm_loss.h"\nint main(void) { printf("%zu %zu %zu %zu\\n", '
                   'sizeof(gemm_loss_args_t), sizeof(gemm_loss_plan_t), offsetof(gemm_loss_args_t, workspace_bytes), '
                   'offsetof(gemm_loss_args_t, teacher_type)); return 0; }\n')
    exe = tmp_path / "s"
    subprocess.run(["gcc", "-I", str(ROOT / "include"), str(src), "-o", str(exe)], check=True)
    got = [int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    assert got == [ctypes.sizeof(dg.GemmLossArgs), ctypes.sizeof(dg.GemmLossPlan), dg.GemmLossArgs.workspace_bytes.offset,
                   dg.GemmLossArgs.teacher_type.offset]


# ---- refusals ---------------------------------------------------------------------------
BASE = 1 << 20   # addresses that are never followed: every call here is refused before a launch


def good(dg, kind=0):
    a = args_of(dg, 16, 64, 32, kind=kind, entries=4)
    a.x, a.w, a.loss, a.lse, a.grad = BASE, 2 * BASE, 3 * BASE, 4 * BASE, 5 * BASE
    a.dx, a.dw = 6 * BASE, 7 * BASE
    a.target = 8 * BASE
    a.teacher_index, a.teacher_logits, a.temperature = 9 * BASE, 10 * BASE, 1.0
    a.workspace, a.workspace_bytes, a.num_cus = 11 * BASE, 0, 256   # too small: the last refusal
    return a


def change(**kw):
    def f(a):
        for k, v in kw.items():
            setattr(a, k, v)
    return f


REFUSED = [   # what, kind, backward too / only, expected status
    ("unknown layout bits", 0, change(layout=0x100), "both", "INVALID"),
    ("layout 2", 0, change(layout=2), "both", "INVALID"),
    ("unknown kind", 0, change(kind=7), "both", "INVALID"),
    ("negative T", 0, change(T=-1), "both", "INVALID"),
    ("no vocabulary", 0, change(V=0), "both", "INVALID"),
    ("no features", 0, change(H=0), "both", "INVALID"),
    ("T too large", 0, change(T=(1 << 24) + 1), "both", "UNSUPPORTED"),
    ("V too large", 0, change(V=(1 << 21) + 8), "both", "UNSUPPORTED"),
    ("H too large", 0, change(H=(1 << 20) + 8), "both", "UNSUPPORTED"),
    ("too many tiles", 0, change(T=1 << 20, V=1 << 18), "both", "UNSUPPORTED"),
    ("too large a dx", 0, change(T=1 << 20, H=1 << 18), "both", "UNSUPPORTED"),
    ("ragged H", 0, change(H=36), "both", "UNSUPPORTED"),
    ("x rows overlap", 0, change(ldx=24), "both", "INVALID"),
    ("x rows unaligned", 0, change(ldx=36), "both", "UNSUPPORTED"),
    ("w rows overlap", 0, change(ldw=24), "both", "INVALID"),
    ("w rows too far apart", 0, change(ldw=(1 << 21) + 8), "both", "UNSUPPORTED"),
    ("x unaligned", 0, change(x=BASE + 8), "both", "UNSUPPORTED"),
    ("w unaligned", 0, change(w=2 * BASE + 2), "both", "UNSUPPORTED"),
    ("no x", 0, change(x=None), "both", "INVALID"),
    ("no w", 0, change(w=None), "both", "INVALID"),
    ("no lse", 0, change(lse=None), "both", "INVALID"),
    ("no target", 0, change(target=None), "both", "INVALID"),
    ("no loss", 0, change(loss=None), "forward", "INVALID"),
    ("no grad", 0, change(grad=None), "backward", "INVALID"),
    ("negative z_loss", 0, change(z_loss=-1.0), "both", "INVALID"),
    ("NaN z_loss", 0, change(z_loss=float("nan")), "both", "INVALID"),
    ("no entries", 1, change(entries=0), "both", "INVALID"),
    ("too many entries", 1, change(entries=1025), "both", "INVALID"),
    ("unknown teacher type", 1, change(teacher_type=3), "both", "INVALID"),
    ("no teacher index", 1, change(teacher_index=None), "both", "INVALID"),
    ("no teacher logits", 1, change(teacher_logits=None), "both", "INVALID"),
    ("temperature 0", 1, change(temperature=0.0), "both", "INVALID"),
    ("temperature NaN", 1, change(temperature=float("nan")), "both", "INVALID"),
    ("temperature inf", 1, change(temperature=float("inf")), "both", "INVALID"),
    ("temperature squared inf", 1, change(temperature=1e20), "both", "INVALID"),
    ("temperature squared 0", 1, change(temperature=1e-30), "both", "INVALID"),
    ("loss over lse", 0, change(loss=4 * BASE + 60), "forward", "INVALID"),
    ("unknown dw type", 0, change(dw_type=3), "both", "INVALID"),
    ("dx unaligned", 0, change(dx=6 * BASE + 8), "backward", "UNSUPPORTED"),
    ("dw unaligned", 0, change(dw=7 * BASE + 4), "backward", "UNSUPPORTED"),
    ("dx rows overlap", 0, change(lddx=8), "backward", "INVALID"),
    ("dw rows unaligned", 0, change(lddw=36), "backward", "UNSUPPORTED"),
    ("dx over x", 0, change(dx=BASE + 64), "backward", "INVALID"),
    ("dw over w", 0, change(dw=2 * BASE), "backward", "INVALID"),
    ("dw over dx", 0, change(dw=6 * BASE + 512), "backward", "INVALID"),
    ("workspace unaligned", 0, change(workspace=11 * BASE + 16), "both", "INVALID"),
    ("negative num_cus", 0, change(num_cus=-1), "both", "INVALID"),
    ("too many CUs", 0, change(num_cus=65537), "both", "INVALID"),
    ("workspace too small", 0, change(), "both", "WORKSPACE"),
    ("workspace too small", 1, change(), "both", "WORKSPACE"),
]


@pytest.mark.parametrize("case", REFUSED, ids=lambda c: f"{c[0]}-{c[1]}")
def test_refused_calls(dg, case):
    what, kind, f, where, status = case
    for name, call in (("forward", dg.gemm_loss_forward), ("backward", dg.gemm_loss_backward)):
        if where not in ("both", name):
            continue
        a = good(dg, kind)
        f(a)
        assert call(a) == getattr(dg, "GEMM_ERR_" + status), (name, dg.gemm_last_error())
        assert dg.gemm_last_error() != ""


def test_kn_needs_whole_chunks_of_the_vocabulary(dg):
    a = good(dg)
    a.layout, a.V = dg.GEMM_B_KN, 60
    assert dg.gemm_loss_forward(a) == dg.GEMM_ERR_UNSUPPORTED
    assert dg.gemm_loss_backward(a) == dg.GEMM_ERR_UNSUPPORTED


def test_nothing_to_do(dg):
    a = good(dg)
    a.T = 0
    assert dg.gemm_loss_forward(a) == dg.GEMM_OK
    b = good(dg)
    b.dx = b.dw = None
    assert dg.gemm_loss_backward(b) == dg.GEMM_OK
    a.dw_type = dg.GEMM_LOSS_DW_FP32_ADD   # nothing is added
    assert dg.gemm_loss_backward(a) == dg.GEMM_OK


def test_null_arguments(dg):
    assert dg._lib.gemm_loss_forward(None) == dg.GEMM_ERR_INVALID
    assert dg._lib.gemm_loss_backward(None) == dg.GEMM_ERR_INVALID
    assert dg._lib.gemm_loss_plan(None, 0, 256, None) == dg.GEMM_ERR_INVALID
    with pytest.raises(dg.GemmError):
        dg.gemm_loss_plan(args_of(dg), False, 0)
    with pytest.raises(dg.GemmError):
        dg.gemm_loss_plan(args_of(dg), True, 65537)


def test_tensor_checks(dg):
    x, w = torch.zeros(4, 16, dtype=torch.bfloat16), torch.zeros(8, 16, dtype=torch.bfloat16)
    t = torch.zeros(4, dtype=torch.int64)
    with pytest.raises(ValueError, match="device tensor"):
        dg.linear_cross_entropy(x, w, t)
    with pytest.raises(TypeError):
        dg.linear_cross_entropy(x.float(), w.float(), t)
    with pytest.raises(TypeError):
        dg.linear_cross_entropy(x, w.half(), t)
    with pytest.raises(ValueError, match="2-D"):
        dg.linear_cross_entropy(x[0], w, t)
