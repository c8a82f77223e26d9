"""The vocabulary losses record nothing for autograd, and say so."""
import warnings

import pytest
import torch

import dense_gemm_work_amd as dg
from loss_util import call_backward, make, on_gpu


def forward(d):
    if "target" in d:
        return dg.linear_cross_entropy(d["x"], d["w"], d["target"])
    return dg.linear_distill(d["x"], d["w"], d["index"], d["logits"])


def cases():
    yield make(4, 16, 16), ("x", "w")
    yield make(4, 16, 16, K=3, kind="distill"), ("x", "w", "logits")


def test_inputs_that_require_gradients_are_warned_about():
    for d, names in cases():   # host tensors: refused after the warning
        for n in names:
            e = dict(d, **{n: d[n].clone().requires_grad_()})
            with pytest.warns(UserWarning, match="not recorded for autograd"), pytest.raises(ValueError, match="device tensor"):
                forward(e)


def test_no_warning_where_nothing_is_lost():
    for d, names in cases():
        with warnings.catch_warnings():
            warnings.simplefilter("error")
            with pytest.raises(ValueError, match="device tensor"):
                forward(d)
            e = dict(d, **{n: d[n].clone().requires_grad_() for n in names})
            with torch.no_grad(), pytest.raises(ValueError, match="device tensor"):
                forward(e)


@pytest.mark.gpu
def test_the_results_are_the_same_with_the_warning():
    for d, names in cases():
        g = on_gpu(d)
        want = forward(g)
        e = dict(g, **{n: g[n].clone().requires_grad_() for n in names})
        with pytest.warns(UserWarning, match="not recorded for autograd"):
            got = forward(e)
        assert all(torch.equal(a, b) and not b.requires_grad for a, b in zip(want, got))
        with warnings.catch_warnings():   # the backward call is the gradient
            warnings.simplefilter("error")
            dx, dw = call_backward(dg, e, got[1])
        assert all(torch.equal(a, b) for a, b in zip((dx, dw), call_backward(dg, g, want[1])))
