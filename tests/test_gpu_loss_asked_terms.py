"""Gradients of the loss with two bf16 terms of dl asked for: any number of rows
comes as near as few rows do."""
import pytest
import torch

from precision_transformer_gemms_gb300 import lpq
from test_gpu_loss import make
from test_gpu_loss_few import check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("t,d,v", [(5, 64, 300), (128, 72, 255), (129, 64, 9), (300, 128, 700), (777, 256, 3000), (1500, 520, 2049), (2304, 2048, 520)])
@pytest.mark.parametrize("piece", [0, 64, 448])
@pytest.mark.parametrize("ignore", [0.0, 0.4])
def test_gradients(t, d, v, piece, ignore):
    h, w, labels, dloss = make(t, d, v, seed=t, ignore=ignore)
    _, lse = lpq.linear_cross_entropy(h, w, labels)
    grads = lambda fp32: lpq.linear_cross_entropy_backward(h, w, labels, lse, dloss, out_fp32=fp32, vocab_piece=piece, two_terms=True)
    dh, dw = grads(True)
    check(h, w, labels, lse, dloss, dh, dw)
    # bf16 results are these, rounded once
    for got, want in zip(grads(False), (dh, dw)):
        assert torch.equal(got, want.bfloat16())
    assert lpq.device_status() == 0


def test_few_rows_are_the_same_either_way():
    h, w, labels, dloss = make(100, 128, 900, ignore=0.2)
    _, lse = lpq.linear_cross_entropy(h, w, labels)
    for a, b in zip(lpq.linear_cross_entropy_backward(h, w, labels, lse, dloss, out_fp32=True),
                    lpq.linear_cross_entropy_backward(h, w, labels, lse, dloss, out_fp32=True, two_terms=True)):
        assert torch.equal(a, b)
