"""GPU tests of the distillation loss's teacher at temperatures below 1: finite
logits stay finite however large they are."""
import pytest
import torch

from loss_util import call_backward, call_forward, make, on_gpu

pytestmark = pytest.mark.gpu
LOWEST, LARGEST = torch.finfo(torch.float32).min, torch.finfo(torch.float32).max


@pytest.fixture(scope="module")
def dg():
    import dense_gemm_work_amd as dg

    assert torch.cuda.is_available(), "GPU test run without a visible GPU"
    return dg


def results(dg, d, tau):
    g = on_gpu(d)
    loss, lse = call_forward(dg, g, tau=tau)
    return (loss, lse) + call_backward(dg, g, lse, tau=tau)


@pytest.mark.parametrize("tau", [0.25, 0.5, 1.0, 2.0])
@pytest.mark.parametrize("T", [7, 200])
def test_rows_of_one_value_are_uniform(dg, T, tau):
    # a softmax does not change with a constant added to its row, whatever the constant
    d = make(T, 700, 64, K=6, kind="distill", ignored=0.0)
    d["logits"].fill_(0.0)
    want = results(dg, d, tau)
    assert torch.isfinite(want[0]).all() and (want[0] > 0).all()
    for value in (LOWEST, LARGEST, -1e38, 2.5e38):
        d["logits"].fill_(value)
        for got, w in zip(results(dg, d, tau), want):
            assert torch.equal(got, w), value


@pytest.mark.parametrize("tau", [0.25, 0.5, 1.0, 2.0])
def test_masked_by_the_lowest_value(dg, tau):
    # entries at the lowest value beside ordinary ones have no weight, as -infinity has not
    d = make(70, 700, 64, K=6, kind="distill", ignored=0.0)
    d["logits"][:, 2] = -float("inf")
    d["logits"][:, 5] = -float("inf")
    want = results(dg, d, tau)
    d["logits"][:, 2] = LOWEST
    d["logits"][:, 5] = LOWEST
    for got, w in zip(results(dg, d, tau), want):
        assert torch.equal(got, w)


@pytest.mark.parametrize("tau", [0.25, 0.5, 1.0, 2.0])
def test_the_largest_value_takes_the_row(dg, tau):
    d = make(70, 700, 64, K=6, kind="distill", ignored=0.0)
    one = dict(d, logits=torch.full((70, 6), -float("inf")))
    one["logits"][:, 1] = 0.0
    want = results(dg, one, tau)
    d["logits"][:, 1] = LARGEST
    for got, w in zip(results(dg, d, tau), want):
        assert torch.equal(got, w)


def test_a_row_of_minus_infinity_has_no_target_at_any_temperature(dg):
    d = make(9, 300, 64, K=4, kind="distill", ignored=0.0)
    d["logits"][3] = -float("inf")
    for tau in (0.25, 1.0, 4.0):
        loss, lse, dx, dw = results(dg, d, tau)
        assert loss[3].item() == 0.0 and not dx[3].any() and (loss[:3] > 0).all()
