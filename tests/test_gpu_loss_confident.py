"""The loss of tokens whose label stands far above the other words.

The logits here are exact: every product is a multiple of 1/64 and every sum
stays below 2^12 of them times 64, so FP32 holds all partial sums.  What is left
are the exponentials (2^-22 of each), the sums' roundings (2^-24 each, some up
and some down) and the last rounding: 2^-21 (1 + |lse|) of lse, and of the loss,
which is log(sum of exp(l - l[label])) and not a difference of two large numbers,
2^-21 (1 + loss).  No such loss is negative: its sum begins with exp(0) = 1.

Gradients: p = exp(l - lse) is off by 2^-21 of itself and the rounding of its
argument, 2^-22 |l - lse|; dl is held in 16 bits; the products' sums are cut by
2^-23 every 16 products."""
import pytest
import torch

from precision_transformer_gemms_gb300 import lpq

pytestmark = pytest.mark.gpu


def make(t, v, ups, seed=0, noise=64):
    """Rows i with logits of size 1 and ups[i % len] added to the label's, by a column of the row's own."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    h = torch.zeros(t, noise + t, device="cuda")
    w = torch.zeros(v, noise + t, device="cuda")
    h[:, :noise] = torch.randint(-3, 4, (t, noise), generator=g, device="cuda") / 8
    w[:, :noise] = torch.randint(-8, 9, (v, noise), generator=g, device="cuda") / 8
    labels = torch.randperm(v, generator=g, device="cuda")[:t]
    up = torch.tensor([ups[i % len(ups)] for i in range(t)], device="cuda").float()
    rows = torch.arange(t, device="cuda")
    h[rows, noise + rows] = 1.0
    w[labels, noise + rows] = up
    return h.bfloat16(), w.bfloat16(), labels


def exact(h, w, labels):
    l = h.double() @ w.double().T
    at = l.gather(1, labels[:, None])
    return l, torch.logsumexp(l, 1), (l - at).exp().sum(1).log()


@pytest.mark.parametrize("v", [200, 1009, 32001, 131072])
def test_loss(v):
    h, w, labels = make(128, v, (0, 10, 12, 16, 20, 24, 26, 28, 30, 45, 60))
    loss, lse = lpq.linear_cross_entropy(h, w, labels)
    _, lse64, loss64 = exact(h, w, labels)
    assert (loss >= 0).all()
    assert ((lse.double() - lse64).abs() <= 2.0 ** -21 * (1 + lse64.abs())).all()
    assert ((loss.double() - loss64).abs() <= 2.0 ** -21 * (1 + loss64)).all()


def test_logits_of_any_size():
    """exp(l - top) has no scale of its own: near the ends of FP32's range too."""
    for size in (2.0 ** 60, 2.0 ** 127):
        h = torch.zeros(2, 8, device="cuda").bfloat16()
        w = torch.zeros(300, 8, device="cuda").bfloat16()
        h[0, 0], h[1, 0] = 1.9921875, -1.9921875
        w[:, 0] = size
        for sign in (1.0, -1.0):
            loss, lse = lpq.linear_cross_entropy(h * sign, w, torch.tensor([5, 299], device="cuda"))
            want = h[:, 0].double() * sign * size
            assert torch.allclose(lse.double(), want, rtol=2.0 ** -22, atol=0)
            assert torch.allclose(loss, torch.full_like(loss, 300.0).log(), rtol=2.0 ** -21, atol=0)


@pytest.mark.parametrize("t", [64, 128])
def test_gradients(t):
    v = 1009
    h, w, labels = make(t, v, (10, 12, 16, 20, 28, 40, 60))
    _, lse = lpq.linear_cross_entropy(h, w, labels)
    dloss = torch.full((t,), 1.0 / 64, device="cuda")
    dh, dw = lpq.linear_cross_entropy_backward(h, w, labels, lse, dloss, out_fp32=True)
    l, _, _ = exact(h, w, labels)
    gap = l - lse.double()[:, None]
    p = gap.exp()
    dl = p.scatter_add(1, labels[:, None], -torch.ones(t, 1, device="cuda", dtype=torch.float64)) / 64
    off = 2.0 ** -16 * dl.abs() + p / 64 * (2.0 ** -21 + 2.0 ** -22 * gap.abs())
    cut = lambda n: (n / 16 + 32) * 2.0 ** -23
    for got, want, tol in ((dh, dl @ w.double(), (off + cut(v) * dl.abs()) @ w.double().abs()),
                           (dw, dl.T @ h.double(), (off + cut(2 * t) * dl.abs()).T @ h.double().abs())):
        assert ((got.double() - want).abs() <= tol + 1e-30).all()
