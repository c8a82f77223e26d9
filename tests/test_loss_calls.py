"""The vocabulary losses' C calls on the host alone: the built library on a HIP
runtime that only records (tests/fake_hip.cpp)."""
import subprocess
from pathlib import Path

import pytest

ROOT = Path(__file__).resolve().parent.parent
PKG = ROOT / "dense_gemm_work_amd"


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    import dense_gemm_work_amd  # noqa: F401  (the library is there)

    exe = tmp_path_factory.mktemp("fake_hip") / "fake_hip"
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-pthread", "-rdynamic", f"-I{ROOT / 'include'}",
                    str(ROOT / "tests" / "fake_hip.cpp"), f"-L{PKG}", "-ldgw_gemm", f"-Wl,-rpath,{PKG}",
                    "-Wl,--allow-shlib-undefined", "-o", str(exe)], check=True)
    return exe


def test_torchs_default_stream_is_named_as_such():
    import dense_gemm_work_amd as dg

    class Stream:
        cuda_stream = 0

    assert dg.stream_word(Stream) == dg.GEMM_NULL_STREAM
    assert dg.GemmLossArgs(stream=dg.stream_word(Stream)).stream == dg.GemmArgs(stream=2 ** 64 - 1).stream is not None
    Stream.cuda_stream = 0x5000
    assert dg.stream_word(Stream) == 0x5000


@pytest.mark.parametrize("scenario", ["release", "two_threads", "streams", "no_exceptions"])
def test_calls(program, scenario):
    res = subprocess.run([str(program), scenario], capture_output=True, text=True, timeout=60)
    assert res.returncode == 0 and res.stdout.split() == ["ok"], res.stdout + res.stderr


# ---- buffers that share memory -------------------------------------------------------------
BASE = 1 << 24   # addresses that are never followed: every call here is refused before a launch
T, V, H, K = 48, 64, 32, 4


def args(dg, kind, backward):
    a = dg.GemmLossArgs(T=T, V=V, H=H, layout=dg.GEMM_B_NK | dg.GEMM_BF16, kind=kind, entries=K, temperature=1.0,
                        ignore_index=-100, num_cus=256)
    names = ["x", "w", "lse", "workspace"] + (["target"] if kind == 0 else ["teacher_index", "teacher_logits"])
    names += ["grad", "dx", "dw"] if backward else ["loss"]
    for i, n in enumerate(names):
        setattr(a, n, (i + 1) * BASE)
    a.workspace_bytes = 1 << 22
    return a, names


def size(dg, a, name, backward):
    if name == "workspace":
        return dg.gemm_loss_plan(a, backward, 256).workspace_bytes
    return {"x": T * H * 2, "w": V * H * 2, "target": T * 8, "teacher_index": T * K * 8, "teacher_logits": T * K * 4,
            "loss": T * 4, "lse": T * 4, "grad": T * 4, "dx": T * H * 2, "dw": V * H * 2}[name]


def status(dg, a, backward):
    return (dg.gemm_loss_backward if backward else dg.gemm_loss_forward)(a)


@pytest.mark.parametrize("kind", [0, 1], ids=["xent", "distill"])
@pytest.mark.parametrize("backward", [False, True], ids=["forward", "backward"])
def test_what_a_call_writes_is_apart_from_all_else(backward, kind):
    import dense_gemm_work_amd as dg

    a, names = args(dg, kind, backward)
    written = {"workspace", "dx", "dw"} if backward else {"workspace", "loss", "lse"}
    step = 256   # keeps every buffer's alignment
    for one in names:
        for two in names:
            if one == two or one not in written:
                continue
            # `two` starts inside `one`, at its start and in its last 256 bytes, and `one` inside `two`
            n1, n2 = size(dg, a, one, backward), size(dg, a, two, backward)
            for move, to in ((two, getattr(a, one)), (two, getattr(a, one) + (n1 - 1) // step * step),
                             (one, getattr(a, two) + (n2 - 1) // step * step)):
                b, _ = args(dg, kind, backward)
                setattr(b, move, to)
                assert status(dg, b, backward) == dg.GEMM_ERR_INVALID, (one, two, hex(to))
                assert "overlap" in dg.gemm_last_error(), (one, two, dg.gemm_last_error())
    # buffers that touch are apart (the workspace, too small here, is the last refusal)
    b, _ = args(dg, kind, backward)
    for one, two in zip(names, names[1:]):
        setattr(b, two, getattr(b, one) + -(-size(dg, a, one, backward) // step) * step)
    b.workspace_bytes = 0
    assert status(dg, b, backward) == dg.GEMM_ERR_WORKSPACE, dg.gemm_last_error()


def test_inputs_may_share_memory():
    import dense_gemm_work_amd as dg

    a, _ = args(dg, 0, True)
    a.w = a.x
    a.grad = a.lse
    a.workspace_bytes = 0
    assert dg.gemm_loss_backward(a) == dg.GEMM_ERR_WORKSPACE, dg.gemm_last_error()


def test_rows_that_lie_between_rows_do_not_overlap():
    # x and dx as halves of one [T, 2H] buffer, w and dw of one [V, 3H]
    import dense_gemm_work_amd as dg

    def call(**kw):
        a, _ = args(dg, 0, True)
        a.ldx = a.lddx = 2 * H
        a.ldw = a.lddw = 3 * H
        a.dx, a.dw = a.x + 2 * H, a.w + 2 * 2 * H
        a.workspace_bytes = 0
        for k, v in kw.items():
            setattr(a, k, v(a) if callable(v) else v)
        return dg.gemm_loss_backward(a)

    assert call() == dg.GEMM_ERR_WORKSPACE, dg.gemm_last_error()
    assert call(dx=lambda a: a.x - 2 * H) == dg.GEMM_ERR_WORKSPACE, dg.gemm_last_error()
    assert call(dw=lambda a: a.w + 2 * H + 3 * 2 * H * 5) == dg.GEMM_ERR_WORKSPACE, dg.gemm_last_error()
    assert call(dx=lambda a: a.x + 2 * H - 16) == dg.GEMM_ERR_INVALID
    assert call(dx=lambda a: a.x + 2 * H + 16) == dg.GEMM_ERR_INVALID
    assert call(dw=lambda a: a.w + 2 * H - 16) == dg.GEMM_ERR_INVALID
    assert call(dw=lambda a: a.w + 2 * 2 * H + 16) == dg.GEMM_ERR_INVALID
    assert call(lddx=2 * H + 8) == dg.GEMM_ERR_INVALID                       # strides that drift apart
    assert call(dw_type=dg.GEMM_LOSS_DW_FP32) == dg.GEMM_ERR_INVALID        # fp32 rows are twice as long
