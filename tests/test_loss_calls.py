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


@pytest.mark.parametrize("scenario", ["release", "two_threads", "streams"])
def test_calls(program, scenario):
    res = subprocess.run([str(program), scenario], capture_output=True, text=True, timeout=60)
    assert res.returncode == 0 and res.stdout.split() == ["ok"], res.stdout + res.stderr
