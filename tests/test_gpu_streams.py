"""Which stream the torch-facing calls run on when the thread has a stream of its own
(gemm_set_stream): torch's current one, also where that is the default stream, whose
handle is 0."""
import pytest
import torch

from loss_util import call_backward, call_forward, make, on_gpu, say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dg():
    import dense_gemm_work_amd as dg

    assert torch.cuda.is_available(), "GPU test run without a visible GPU"
    return dg


def test_calls_on_the_default_stream_while_the_threads_is_busy(dg):
    loss_in = on_gpu(make(300, 2000, 136, seed=3))
    kd_in = on_gpu(make(300, 2000, 136, K=8, kind="distill", seed=4))
    a, b = loss_in["x"], loss_in["w"]

    def run():
        out = []
        for g in (loss_in, kd_in):
            loss, lse = call_forward(dg, g)
            out += [loss, lse, *call_backward(dg, g, lse)]
        c, one = torch.empty(300, 2000, device="cuda:0"), torch.empty(300, 2000, device="cuda:0")
        dg.gemm_tensors(a, b, c, b_layout="nk")
        dg.gemm_grouped_tensors([(a, b, one)], b_layout="nk")
        return out + [c, one, dg.matmul(a, b, b_layout="nk")]

    want = run()
    side = torch.cuda.Stream()
    big = torch.randn(8192, 8192, device="cuda:0").bfloat16()
    big @ big
    torch.cuda.synchronize()
    say("  the thread's stream gets 100 products to do")
    try:
        dg.gemm_set_stream(side.cuda_stream)
        with torch.cuda.stream(side):
            for _ in range(100):
                big @ big
        got = run()
        done = torch.cuda.Event()
        done.record()
        done.synchronize()
        busy = not side.query()
    finally:
        dg.gemm_set_stream(None)
    torch.cuda.synchronize()
    assert busy, "the calls waited for the thread's stream, or it had too little to do"
    assert all(torch.equal(x, y) for x, y in zip(got, want))
