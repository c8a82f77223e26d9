"""GPU test of the vocabulary losses on rows of operands and results that lie in turn
in one buffer."""
import pytest
import torch

from loss_util import call_backward, call_forward, make, on_gpu, to_layout

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("layout", ["nk", "kn"])
@pytest.mark.parametrize("T", [5, 100, 700], ids=lambda t: f"T{t}")
def test_operands_and_results_in_one_buffer(T, layout):
    import dense_gemm_work_amd as dg

    V, H = 1000, 136
    g = on_gpu(make(T, V, H, seed=9))
    w = to_layout(g["w"], layout)
    loss, lse = call_forward(dg, g, layout)
    want = call_backward(dg, g, lse, layout)
    rows, cols = w.shape
    xs = torch.full((T, 2 * H), 7.0, dtype=torch.bfloat16, device="cuda:0")
    ws = torch.full((rows, 2 * cols + 8), 7.0, dtype=torch.bfloat16, device="cuda:0")
    xs[:, :H] = g["x"]
    ws[:, cols + 8:] = w
    g["x"] = xs[:, :H]
    l2, e2 = call_forward(dg, g, layout, w=ws[:, cols + 8:])
    call_backward(dg, g, lse, layout, w=ws[:, cols + 8:], dx=xs[:, H:], dw=ws[:, :cols])
    assert torch.equal(l2, loss) and torch.equal(e2, lse)
    assert torch.equal(xs[:, H:], want[0]) and torch.equal(ws[:, :cols], want[1])
    assert torch.equal(xs[:, :H], on_gpu(make(T, V, H, seed=9))["x"]) and torch.equal(ws[:, cols + 8:], w)
    assert bool((ws[:, cols: cols + 8] == 7.0).all())
