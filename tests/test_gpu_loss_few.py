"""Gradients of the loss over few rows (up to 128), FP32: dl in two bf16 terms
leaves at most 2^-16 of each value out.  To that come the cuts of the FP32 sums,
2^-23 of the running sum per 16 products, doubled here: in the logits (their
absolute error is dl's relative one), and in the products' sums."""
import pytest
import torch

from precision_transformer_gemms_gb300 import lpq
from test_gpu_loss import make

pytestmark = pytest.mark.gpu


def reference(h, w, labels, lse, dloss):
    h, w = h.double(), w.double()
    logits = h @ w.T
    dl = (logits - lse.double()[:, None]).exp()
    target = (labels >= 0) & (labels < w.shape[0])
    rows = torch.arange(h.shape[0], device="cuda")[target]
    dl[rows, labels[target]] -= 1
    dl = torch.where(target[:, None], dl * dloss.double()[:, None], 0.0)
    # p itself, against which the label's 1 - p may be small
    size = dl.abs()
    size[rows, labels[target]] += 2 * dloss.double().abs()[target]
    cuts = logits.abs().max() * h.shape[1] / 16 * 2.0**-22
    return dl @ w, size @ w.abs(), dl.T @ h, size.T @ h.abs(), 2.0**-16 + float(cuts)


def check(h, w, labels, lse, dloss, dh, dw):
    want_h, size_h, want_w, size_w, eps = reference(h, w, labels, lse, dloss)
    t, v = h.shape[0], w.shape[0]
    assert ((dh.double() - want_h).abs() <= size_h * (eps + v / 16 * 2.0**-22) + 1e-30).all()
    assert ((dw.double() - want_w).abs() <= size_w * (eps + (2 * t / 16 + 8) * 2.0**-22) + 1e-30).all()


@pytest.mark.parametrize("t", [1, 2, 31, 32, 33, 63, 64, 65, 127, 128])
@pytest.mark.parametrize("d,v", [(64, 9), (72, 255), (256, 1000), (520, 2049)])
def test_gradients(t, d, v):
    h, w, labels, dloss = make(t, d, v, seed=t, ignore=0.0)
    _, lse = lpq.linear_cross_entropy(h, w, labels)
    check(h, w, labels, lse, dloss, *lpq.linear_cross_entropy_backward(h, w, labels, lse, dloss, out_fp32=True))
    assert lpq.device_status() == 0


@pytest.mark.parametrize("t", [5, 100])
@pytest.mark.parametrize("piece", [64, 448])
def test_pieces_and_rows_without_target(t, piece):
    h, w, labels, dloss = make(t, 192, 1500, seed=t, ignore=0.5)
    _, lse = lpq.linear_cross_entropy(h, w, labels)
    got = lpq.linear_cross_entropy_backward(h, w, labels, lse, dloss, out_fp32=True, vocab_piece=piece)
    check(h, w, labels, lse, dloss, *got)


def test_closer_than_one_term():
    """At 128 rows an order of magnitude closer than at 129, where dl is one bf16."""
    def off(t):
        h, w, labels, dloss = make(t, 128, 600, seed=7, ignore=0.0)
        _, lse = lpq.linear_cross_entropy(h, w, labels)
        _, dw = lpq.linear_cross_entropy_backward(h, w, labels, lse, dloss, out_fp32=True)
        want = reference(h, w, labels, lse, dloss)[2]
        return float((dw.double() - want).norm() / want.norm())

    assert off(128) < 2.0**-15 and off(128) < 0.1 * off(129)


def test_infinite_dloss_stays_an_infinity_or_nan():
    """What the other rows get is theirs: an infinite dloss spoils its own row of dh, not the others."""
    h, w, labels, dloss = make(6, 64, 100, ignore=0.0)
    _, lse = lpq.linear_cross_entropy(h, w, labels)
    dloss[2] = float("inf")
    dh, _ = lpq.linear_cross_entropy_backward(h, w, labels, lse, dloss, out_fp32=True)
    assert not dh[2].isfinite().any()
    keep = torch.arange(6, device="cuda") != 2
    want_h, size_h, _, _, eps = reference(h[keep], w, labels[keep], lse[keep], dloss[keep])
    assert ((dh[keep].double() - want_h).abs() <= size_h * (eps + 100 / 16 * 2.0**-22) + 1e-30).all()
