"""Every kernel of the feed-forward block and the adapters is one that some call launches."""
import subprocess
from pathlib import Path

ROOT = Path(__file__).resolve().parent.parent
PKG = ROOT / "dense_gemm_work_amd"


def test_every_kernel_is_reached(tmp_path):
    import dense_gemm_work_amd  # noqa: F401  (the library is there)

    exe = tmp_path / "reach"
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Wno-unused-function", "-pthread", "-rdynamic", f"-I{ROOT / 'include'}",
                    str(ROOT / "tests" / "fake_hip_reach.cpp"), f"-L{PKG}", "-ldgw_gemm", f"-Wl,-rpath,{PKG}",
                    "-Wl,--allow-shlib-undefined", "-o", str(exe)], check=True)
    res = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert res.returncode == 0, res.stdout + res.stderr
    assert not res.stdout, "no call reaches:\n" + res.stdout
