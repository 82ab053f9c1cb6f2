"""The loss's backward pass with many rows that have no target: any share and
place of them, whatever they hold, both ways of joining dh, pieces included."""
import pytest
import torch

from precision_transformer_gemms_gb300 import lpq
from test_gpu_loss import check_grads, make

pytestmark = pytest.mark.gpu


def share(labels, keep, seed=3):
    """Leaves `keep` rows with a target, at random places."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    gone = torch.randperm(labels.numel(), generator=g, device="cuda")[keep:]
    labels[gone] = -100
    return gone


@pytest.mark.parametrize("t,d,v", [(300, 128, 700), (1500, 256, 3000), (2304, 2048, 520)])
@pytest.mark.parametrize("keep", [0, 1, 63, 64, 65, 127, 128, 255, 256, 257, 299])
@pytest.mark.parametrize("fp32", [False, True])
def test_any_number_of_rows_with_a_target(t, d, v, keep, fp32):
    h, w, labels, dloss = make(t, d, v, seed=keep, ignore=0.0)
    gone = share(labels, keep)
    _, lse = lpq.linear_cross_entropy(h, w, labels)
    want = h.clone()
    want[gone] = 0
    # the other rows hold no numbers at all
    h[gone] = float("nan")
    dloss[gone] = float("inf")
    lse[gone] = float("nan")
    dh, dw = lpq.linear_cross_entropy_backward(h, w, labels, lse, dloss, out_fp32=fp32)
    assert not dh[gone].any()
    dloss[gone], lse[gone] = 0.0, 1.0
    check_grads(want, w, labels, lse, dloss, dh, dw)
    assert lpq.device_status() == 0


@pytest.mark.parametrize("piece", [64, 320, 1024])
@pytest.mark.parametrize("keep", [10, 400])
def test_pieces(piece, keep):
    h, w, labels, dloss = make(500, 192, 1500, ignore=0.0)
    gone = share(labels, keep)
    _, lse = lpq.linear_cross_entropy(h, w, labels)
    h[gone] = float("inf")
    got = lpq.linear_cross_entropy_backward(h, w, labels, lse, dloss, vocab_piece=piece)
    h[gone] = 0
    check_grads(h, w, labels, lse, dloss, *got)


def test_same_bits_as_the_rows_alone():
    """The gradients of the rows with a target are those of a call without the others."""
    h, w, labels, dloss = make(900, 256, 2000, ignore=0.0)
    share(labels, 512)
    valid = labels >= 0
    _, lse = lpq.linear_cross_entropy(h, w, labels)
    dh, dw = lpq.linear_cross_entropy_backward(h, w, labels, lse, dloss, out_fp32=True)
    dh1, dw1 = lpq.linear_cross_entropy_backward(h[valid].contiguous(), w, labels[valid].contiguous(), lse[valid].contiguous(),
                                                 dloss[valid].contiguous(), out_fp32=True)
    assert torch.equal(dw, dw1)
    assert torch.allclose(dh[valid], dh1, rtol=1e-5, atol=1e-9)  # (dh's sum may be split differently)


def test_more_rows_than_one_count():
    """Rows beyond the counting CTA's 1024 at a time."""
    h, w, labels, dloss = make(5000, 64, 300, ignore=0.6)
    _, lse = lpq.linear_cross_entropy(h, w, labels)
    check_grads(h, w, labels, lse, dloss, *lpq.linear_cross_entropy_backward(h, w, labels, lse, dloss))
