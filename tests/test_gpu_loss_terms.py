"""Gradients of the loss with dl in two bf16 terms: where few rows have a target,
however many there are beside them."""
import pytest
import torch

from precision_transformer_gemms_gb300 import lpq
from test_gpu_loss import check_grads, make
from test_gpu_loss_few import check
from test_gpu_loss_rows import share

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("t,d,v", [(129, 64, 300), (512, 128, 700), (1500, 256, 3000), (2304, 2048, 520)])
@pytest.mark.parametrize("keep", [1, 20, 64, 65, 127, 128])
@pytest.mark.parametrize("piece", [0, 256])
def test_few_rows_with_a_target_among_many(t, d, v, keep, piece):
    """As near as a call of those rows alone would come (tests of few rows)."""
    h, w, labels, dloss = make(t, d, v, seed=keep, ignore=0.0)
    gone = share(labels, keep)
    _, lse = lpq.linear_cross_entropy(h, w, labels)
    h[gone], dloss[gone], lse[gone] = float("nan"), float("inf"), float("nan")
    dh, dw = lpq.linear_cross_entropy_backward(h, w, labels, lse, dloss, out_fp32=True, vocab_piece=piece)
    assert not dh[gone].any()
    kept = labels >= 0
    check(h[kept], w, labels[kept], lse[kept], dloss[kept], dh[kept], dw)
    dh, dw = lpq.linear_cross_entropy_backward(h, w, labels, lse, dloss, vocab_piece=piece)
    h[gone], dloss[gone], lse[gone] = 0.0, 0.0, 1.0
    check_grads(h, w, labels, lse, dloss, dh, dw)
    assert lpq.device_status() == 0
