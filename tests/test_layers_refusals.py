"""Calls of the feed-forward block, the adapters and the losses that must be refused, on the host alone:
nothing is launched, and no address is followed."""
import pytest

from test_layers_calls import BASE, F, H, Ffn, L, Lora, N, R, T, good

EMPTY = [   # kind, what is written, what it would overwrite, "+ n": that many bytes into it
    (Ffn, "dw_gate", "w_gate", 0), (Ffn, "dw_up", "w_down", 0), (Ffn, "dw_down", "w_up", H * 2 * 8), (Ffn, "dw_gate", "dw_up", 0),
    (Lora, "da", "a", 0), (Lora, "db", "w", 0), (Lora, "db", "b", R * 2 * 8), (Lora, "da", "db", 0), (Lora, "da", "scale", 0),
]


@pytest.fixture(scope="module")
def dg():
    import dense_gemm_work_amd as dg

    return dg


@pytest.mark.parametrize("case", EMPTY, ids=lambda c: f"{c[1]}-{c[2]}")
def test_no_rows_overwrite_nothing(dg, case):
    # the gradients of no rows are zeros: written, and so apart from all else that the call takes
    kind, one, two, more = case
    a, _ = good(dg, kind, True)
    a.T = 0
    setattr(a, one, getattr(a, two) + more)
    assert kind.call(dg, a, True) == dg.GEMM_ERR_INVALID, dg.gemm_last_error()
    assert "overlap" in dg.gemm_last_error()


def test_no_rows_of_a_loss_overwrite_nothing(dg):
    a = dg.GemmLossArgs(T=0, V=F, H=H, layout=dg.GEMM_B_NK | dg.GEMM_BF16, kind=dg.GEMM_LOSS_XENT, num_cus=256)
    a.x, a.w, a.dx, a.dw = BASE, 2 * BASE, 3 * BASE, 2 * BASE + 128
    assert dg.gemm_loss_backward(a) == dg.GEMM_ERR_INVALID and "overlap" in dg.gemm_last_error()


STRIDES = ["ldx", "ldw_gate", "ldw_up", "ldw_down", "ldgate", "ldup"], ["lddy", "lddx", "lddw_gate", "lddw_up", "lddw_down"]


@pytest.mark.parametrize("fp32", [False, True])
def test_strides_whose_bytes_pass_64_bits(dg, fp32):
    # 2^62 elements of four bytes and 2^63 of two are no bytes at all
    for backward in (False, True):
        for name in STRIDES[0] + (STRIDES[1] if backward else ["ldy"]):
            row = F if name in ("ldw_down", "lddw_down", "ldgate", "ldup") else H
            for ld, status in ((2 ** 62 + row, "UNSUPPORTED"), (2 ** 63 - 2 ** 10, "UNSUPPORTED"), (row - 2 ** 63, "INVALID"), (-row, "INVALID")):
                a, _ = good(dg, Ffn, backward)
                a.dw_type = int(fp32)
                setattr(a, name, ld)
                a.workspace_bytes = 0   # a stride that gets through ends here, not in a launch
                assert Ffn.call(dg, a, backward) == getattr(dg, "GEMM_ERR_" + status), (name, ld, dg.gemm_last_error())
