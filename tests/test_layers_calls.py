"""The C calls of the feed-forward block and the adapters on the host alone: a HIP
runtime that only records, refusals, and buffers that share memory."""
import subprocess
from pathlib import Path

import pytest

ROOT = Path(__file__).resolve().parent.parent
PKG = ROOT / "dense_gemm_work_amd"
BASE = 1 << 24   # addresses that are never followed: every call here is refused before a launch
T, H, F, N, R, L = 48, 64, 96, 128, 8, 3


@pytest.fixture(scope="module")
def dg():
    import dense_gemm_work_amd as dg

    return dg


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    import dense_gemm_work_amd  # noqa: F401  (the library is there)

    exe = tmp_path_factory.mktemp("fake_hip_layers") / "fake_hip_layers"
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Wno-unused-function", "-pthread", "-rdynamic", f"-I{ROOT / 'include'}",
                    str(ROOT / "tests" / "fake_hip_layers.cpp"), f"-L{PKG}", "-ldgw_gemm", f"-Wl,-rpath,{PKG}",
                    "-Wl,--allow-shlib-undefined", "-o", str(exe)], check=True)
    return exe


@pytest.mark.parametrize("scenario", ["stream", "workspace", "no_exceptions"])
def test_calls(program, scenario):
    res = subprocess.run([str(program), scenario], capture_output=True, text=True, timeout=60)
    assert res.returncode == 0 and res.stdout.split() == ["ok"], res.stdout + res.stderr


class Ffn:
    names = ["x", "w_gate", "w_up", "w_down", "gate", "up", "workspace"]
    size = {"x": T * H, "w_gate": F * H, "w_up": F * H, "w_down": H * F, "gate": T * F, "up": T * F, "y": T * H, "dy": T * H,
            "dx": T * H, "dw_gate": F * H, "dw_up": F * H, "dw_down": H * F}

    @staticmethod
    def args(dg):
        return dg.GemmFfnArgs(T=T, H=H, F=F, layout=dg.GEMM_B_NK | dg.GEMM_BF16, num_cus=256, workspace_bytes=1 << 22)

    @staticmethod
    def call(dg, a, backward):
        return (dg.gemm_ffn_backward if backward else dg.gemm_ffn_forward)(a)

    @staticmethod
    def plan(dg, a, backward):
        return dg.gemm_ffn_plan(a, backward, 256)

    written = ({"y", "gate", "up", "workspace"}, {"dx", "dw_gate", "dw_up", "dw_down", "workspace"})
    more = (["y"], ["dy", "dx", "dw_gate", "dw_up", "dw_down"])


class Lora:
    names = ["x", "w", "a", "b", "adapter", "scale", "workspace"]
    size = {"x": T * H, "w": N * H, "a": L * R * H, "b": L * N * R, "adapter": T * 4, "scale": L * 2, "y": T * N, "dy": T * N,
            "dx": T * H, "da": L * R * H, "db": L * N * R}

    @staticmethod
    def args(dg):
        return dg.GemmLoraArgs(T=T, H=H, N=N, R=R, adapters=L, layout=dg.GEMM_B_NK | dg.GEMM_BF16, num_cus=256,
                               workspace_bytes=1 << 23)

    @staticmethod
    def call(dg, a, backward):
        return (dg.gemm_lora_backward if backward else dg.gemm_lora_forward)(a)

    @staticmethod
    def plan(dg, a, backward):
        return dg.gemm_lora_plan(a, backward, 256)

    written = ({"y", "workspace"}, {"dx", "da", "db", "workspace"})
    more = (["y"], ["dy", "dx", "da", "db"])


def good(dg, kind, backward):
    a = kind.args(dg)
    names = kind.names + kind.more[backward]
    for i, n in enumerate(names):
        setattr(a, n, (i + 1) * BASE)
    return a, names


@pytest.mark.parametrize("backward", [False, True], ids=["forward", "backward"])
@pytest.mark.parametrize("kind", [Ffn, Lora], ids=["ffn", "lora"])
def test_what_a_call_writes_is_apart_from_all_else(dg, kind, backward):
    a, names = good(dg, kind, backward)
    size = {n: 2 * s for n, s in kind.size.items()}   # bytes
    size["workspace"] = kind.plan(dg, a, backward).workspace_bytes
    step = 256
    for one in names:
        for two in names:
            if one == two or one not in kind.written[backward]:
                continue
            for move, to in ((two, getattr(a, one)), (two, getattr(a, one) + (size[one] - 1) // step * step),
                             (one, getattr(a, two) + (size[two] - 1) // step * step)):
                b, _ = good(dg, kind, backward)
                setattr(b, move, to)
                assert kind.call(dg, b, backward) == dg.GEMM_ERR_INVALID, (one, two, hex(to))
                assert "overlap" in dg.gemm_last_error(), (one, two, dg.gemm_last_error())
    # buffers that touch are apart (the workspace, too small here, is the last refusal)
    b, _ = good(dg, kind, backward)
    for one, two in zip(names, names[1:]):
        setattr(b, two, getattr(b, one) + -(-size[one] // step) * step)
    b.workspace_bytes = 0
    assert kind.call(dg, b, backward) == dg.GEMM_ERR_WORKSPACE, dg.gemm_last_error()


@pytest.mark.parametrize("kind", [Ffn, Lora], ids=["ffn", "lora"])
def test_inputs_may_share_memory(dg, kind):
    a, _ = good(dg, kind, True)
    if kind is Ffn:
        a.w_up, a.dy, a.up = a.w_gate, a.x, a.gate
    else:
        a.dy = a.x
        a.ldx = a.lddy = N
    a.workspace_bytes = 0
    assert kind.call(dg, a, True) == dg.GEMM_ERR_WORKSPACE, dg.gemm_last_error()


def test_rows_that_lie_between_rows_do_not_overlap(dg):
    # gate and up as halves of one [T, 2F] buffer, w_gate's and w_up's gradients of one [F, 2H]
    a, _ = good(dg, Ffn, False)
    a.ldgate = a.ldup = 2 * F
    a.up = a.gate + 2 * F
    a.workspace_bytes = 0
    assert dg.gemm_ffn_forward(a) == dg.GEMM_ERR_WORKSPACE, dg.gemm_last_error()
    a.up = a.gate + 2 * F - 16
    assert dg.gemm_ffn_forward(a) == dg.GEMM_ERR_INVALID
    b, _ = good(dg, Ffn, True)
    b.lddw_gate = b.lddw_up = 2 * H
    b.dw_up = b.dw_gate + 2 * H
    b.workspace_bytes = 0
    assert dg.gemm_ffn_backward(b) == dg.GEMM_ERR_WORKSPACE, dg.gemm_last_error()


def change(**kw):
    def f(a):
        for k, v in kw.items():
            setattr(a, k, v)
    return f


REFUSED = [   # kind, what, where, status
    (Ffn, change(layout=0x100), "both", "INVALID"),
    (Ffn, change(layout=2), "both", "INVALID"),
    (Ffn, change(act=3), "both", "INVALID"),
    (Ffn, change(T=-1), "both", "INVALID"),
    (Ffn, change(H=0), "both", "INVALID"),
    (Ffn, change(F=0), "both", "INVALID"),
    (Ffn, change(H=36), "both", "UNSUPPORTED"),
    (Ffn, change(F=100), "both", "UNSUPPORTED"),
    (Ffn, change(T=(1 << 24) + 1), "both", "UNSUPPORTED"),
    (Ffn, change(F=(1 << 20) + 8), "both", "UNSUPPORTED"),
    (Ffn, change(T=1 << 20, H=1 << 18), "both", "UNSUPPORTED"),
    (Ffn, change(H=1 << 19, F=1 << 19), "both", "UNSUPPORTED"),
    (Ffn, change(dw_type=3), "both", "INVALID"),
    (Ffn, change(ldx=56), "both", "INVALID"),
    (Ffn, change(ldx=68), "both", "UNSUPPORTED"),
    (Ffn, change(ldw_gate=56), "both", "INVALID"),
    (Ffn, change(ldw_up=(1 << 21) + 8), "both", "UNSUPPORTED"),
    (Ffn, change(ldw_down=100), "both", "UNSUPPORTED"),
    (Ffn, change(ldgate=90), "both", "INVALID"),
    (Ffn, change(ldup=100), "both", "UNSUPPORTED"),
    (Ffn, change(x=BASE + 8), "both", "UNSUPPORTED"),
    (Ffn, change(w_down=4 * BASE + 2), "both", "UNSUPPORTED"),
    (Ffn, change(gate=5 * BASE + 8), "both", "UNSUPPORTED"),
    (Ffn, change(x=None), "both", "INVALID"),
    (Ffn, change(w_up=None), "both", "INVALID"),
    (Ffn, change(y=None), "forward", "INVALID"),
    (Ffn, change(up=None), "forward", "INVALID"),
    (Ffn, change(gate=None), "backward", "INVALID"),
    (Ffn, change(dy=None), "backward", "INVALID"),
    (Ffn, change(lddx=40), "backward", "INVALID"),
    (Ffn, change(lddw_down=100), "backward", "UNSUPPORTED"),
    (Ffn, change(dw_type=1, lddw_down=98), "backward", "UNSUPPORTED"),
    (Ffn, change(dw_gate=10 * BASE + 8), "backward", "UNSUPPORTED"),
    (Ffn, change(workspace=7 * BASE + 16), "both", "INVALID"),
    (Ffn, change(num_cus=-1), "both", "INVALID"),
    (Ffn, change(num_cus=65537), "both", "INVALID"),
    (Ffn, change(workspace_bytes=0), "both", "WORKSPACE"),
    (Lora, change(layout=0x100), "both", "INVALID"),
    (Lora, change(T=-1), "both", "INVALID"),
    (Lora, change(N=0), "both", "INVALID"),
    (Lora, change(R=0), "both", "INVALID"),
    (Lora, change(adapters=0), "both", "INVALID"),
    (Lora, change(R=12), "both", "UNSUPPORTED"),
    (Lora, change(R=1032), "both", "UNSUPPORTED"),
    (Lora, change(N=100), "both", "UNSUPPORTED"),
    (Lora, change(adapters=(1 << 16) + 1), "both", "UNSUPPORTED"),
    (Lora, change(adapters=1 << 16, R=1024, H=1 << 20), "both", "UNSUPPORTED"),
    (Lora, change(T=1 << 20, N=1 << 18), "both", "UNSUPPORTED"),
    (Lora, change(T=1 << 20, adapters=1 << 15), "backward", "UNSUPPORTED"),
    (Lora, change(T=1 << 22, R=1024), "both", "UNSUPPORTED"),
    (Lora, change(adapters=1 << 16, H=1 << 14, stride_a=0, ldx=0, ldw=0, lddx=0), "backward", "UNSUPPORTED"),
    (Lora, change(stride_a=(1 << 40) + 8), "both", "INVALID"),
    (Lora, change(stride_b=1 << 62), "both", "INVALID"),
    (Lora, change(scale=6 * BASE + 2), "both", "UNSUPPORTED"),
    (Lora, change(dab_type=3), "both", "INVALID"),
    (Lora, change(stride_a=R * H - 8), "both", "INVALID"),
    (Lora, change(stride_b=N * R + 4), "both", "INVALID"),
    (Lora, change(ldw=40), "both", "INVALID"),
    (Lora, change(ldy=100), "forward", "INVALID"),
    (Lora, change(lddy=132), "backward", "UNSUPPORTED"),
    (Lora, change(a=3 * BASE + 8), "both", "UNSUPPORTED"),
    (Lora, change(adapter=5 * BASE + 4), "both", "UNSUPPORTED"),
    (Lora, change(adapter=None), "both", "INVALID"),
    (Lora, change(b=None), "both", "INVALID"),
    (Lora, change(y=None), "forward", "INVALID"),
    (Lora, change(dy=None), "backward", "INVALID"),
    (Lora, change(da=10 * BASE + 8), "backward", "UNSUPPORTED"),
    (Lora, change(workspace_bytes=0), "both", "WORKSPACE"),
]


@pytest.mark.parametrize("case", range(len(REFUSED)))
def test_refused_calls(dg, case):
    kind, f, where, status = REFUSED[case]
    for backward, name in ((False, "forward"), (True, "backward")):
        if where in ("both", name):
            a, _ = good(dg, kind, backward)
            f(a)
            assert kind.call(dg, a, backward) == getattr(dg, "GEMM_ERR_" + status), (name, dg.gemm_last_error())
            assert dg.gemm_last_error() != ""


@pytest.mark.parametrize("kind", [Ffn, Lora], ids=["ffn", "lora"])
def test_nothing_to_do(dg, kind):
    a, _ = good(dg, kind, False)
    a.T = 0
    assert kind.call(dg, a, False) == dg.GEMM_OK
    b, _ = good(dg, kind, True)
    for n in ("dx", "dw_gate", "dw_up", "dw_down", "da", "db"):
        if n in kind.more[1]:
            setattr(b, n, None)
    assert kind.call(dg, b, True) == dg.GEMM_OK
    c, _ = good(dg, kind, True)
    c.T = 0
    setattr(c, "dw_type" if kind is Ffn else "dab_type", 2)   # nothing is added
    assert kind.call(dg, c, True) == dg.GEMM_OK


def test_null_arguments(dg):
    for name in ("ffn", "lora"):
        assert getattr(dg._lib, f"gemm_{name}_forward")(None) == dg.GEMM_ERR_INVALID
        assert getattr(dg._lib, f"gemm_{name}_backward")(None) == dg.GEMM_ERR_INVALID
        assert getattr(dg._lib, f"gemm_{name}_plan")(None, 0, 256, None) == dg.GEMM_ERR_INVALID
    for kind in (Ffn, Lora):
        for cus in (0, 65537):
            with pytest.raises(dg.GemmError):
                (dg.gemm_ffn_plan if kind is Ffn else dg.gemm_lora_plan)(kind.args(dg), False, cus)
