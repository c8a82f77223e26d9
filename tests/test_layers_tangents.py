"""Inputs with forward-mode tangents, which the calls do not carry on, are warned about."""
import warnings

import pytest
import torch
from torch.autograd import forward_ad

import ffn_util as fu
import lora_util as lu


@pytest.fixture(scope="module")
def dg():
    import dense_gemm_work_amd as dg

    return dg


def calls(dg):
    """{name: (inputs, call of them)}; every call ends with the refusal of host tensors."""
    d, e = fu.make(4, 16, 24), lu.make(4, 16, 24, 2, 8)
    target = torch.zeros(4, dtype=torch.int64)
    return {
        "ffn": ([d["x"], *(d[w] for w in fu.WEIGHTS)], lambda *t: dg.gated_ffn(*t)),
        "lora": ([e[k] for k in ("x", "w", "a", "b")], lambda *t: dg.linear_lora(*t, e["adapter"])),
        "loss": ([d["x"], d["w_gate"]], lambda *t: dg.linear_cross_entropy(*t, target)),
        "distill": ([d["x"], d["w_gate"], torch.zeros(4, 1)], lambda x, w, q: dg.linear_distill(x, w, target[:, None], q)),
    }


@pytest.mark.parametrize("name", ["ffn", "lora", "loss", "distill"])
def test_tangents_are_warned_about(dg, name):
    inputs, call = calls(dg)[name]
    with forward_ad.dual_level():
        for i, t in enumerate(inputs):
            dual = [forward_ad.make_dual(u, torch.ones_like(u)) if i == j else u for j, u in enumerate(inputs)]
            with pytest.warns(UserWarning, match="tangents of its inputs are dropped"), torch.no_grad():
                with pytest.raises(ValueError, match="device tensor"):
                    call(*dual)
        with warnings.catch_warnings():   # none among them
            warnings.simplefilter("error")
            with pytest.raises(ValueError, match="device tensor"):
                call(*inputs)
