"""The vocabulary cross entropy and its gradients on the GPU against the
formulas in 64 bits.

Tolerances: products of bf16 values are exact in FP32 and the tensor core adds
16 of them at a time, so a sum of n products is off by at most
e(n) = (n / 16 + 32) 2^-23 of the sum of their magnitudes.  A row's lse is off
by its worst logit plus the roundings of the sums over the vocabulary (2^-19,
relative to 1 + |lse|); dl = g (p - 1{label}) is rounded to bf16 (2^-8 of its
size) after p's own error, and bf16 results once more (2^-8)."""
import pytest
import torch

from precision_transformer_gemms_gb300 import lpq

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def e(n):
    return (n / 16 + 32) * 2.0 ** -23


def make(t, d, v, seed=0, ignore=0.1, std=0.05):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    h = torch.randn(t, d, generator=g, device="cuda").to(BF)
    w = (std * torch.randn(v, d, generator=g, device="cuda")).to(BF)
    labels = torch.randint(0, v, (t,), generator=g, device="cuda")
    labels[torch.rand(t, generator=g, device="cuda") < ignore] = -100
    dloss = torch.rand(t, generator=g, device="cuda") / max(t, 1)
    return h, w, labels, dloss


def reference(h, w, labels):
    l = h.double() @ w.double().T
    lse = torch.logsumexp(l, 1)
    valid = (labels >= 0) & (labels < w.shape[0])
    at = l.gather(1, torch.where(valid, labels, 0)[:, None])[:, 0]
    off = e(h.shape[1]) * (h.double().abs() @ w.double().abs().T).amax(1)
    return l, lse, torch.where(valid, lse - at, 0.0), valid, off


def check_loss(h, w, labels, loss, lse):
    l, lse64, loss64, valid, off = reference(h, w, labels)
    tol = off + 2.0 ** -19 * (1 + lse64.abs())
    assert torch.all((lse.double() - lse64).abs() <= tol)
    assert torch.all((loss.double() - loss64).abs() <= torch.where(valid, 2 * tol, 0.0))


def check_grads(h, w, labels, lse, dloss, dh, dw):
    l, _, _, valid, off = reference(h, w, labels)
    p = (l - lse.double()[:, None]).exp()
    one = torch.zeros_like(p)
    one[valid, labels[valid]] = 1.0
    g = torch.where(valid, dloss.double(), 0.0)[:, None]
    dl = g * (p - one)
    dl = torch.where(valid[:, None], dl, 0.0)
    fuzz = 1.01 * 2.0 ** -8 * dl.abs() + g.abs() * p * (off + 2.0 ** -18)[:, None]
    fuzz = torch.where(valid[:, None], fuzz, 0.0)
    t, v = l.shape
    out = 2.0 ** -8 if dh.dtype == BF else 2.0 ** -23
    tiny = 1e-30 * g.abs().max() if t else 0.0
    for got, want, tol in ((dh, dl @ w.double(), (fuzz + e(v) * dl.abs()) @ w.double().abs()),
                           (dw, dl.T @ h.double(), (fuzz + e(t) * dl.abs()).T @ h.double().abs())):
        err = (got.double() - want).abs()
        tol = 1.01 * tol + out * want.abs() + tiny
        assert torch.all(err <= tol), float((err / tol.clamp_min(1e-300)).max())


SHAPES = [(1, 8, 1), (1, 64, 2), (2, 16, 100), (3, 8, 65), (7, 72, 257), (33, 512, 1009), (64, 64, 64), (127, 128, 383), (129, 136, 1000), (255, 256, 511),
          (256, 256, 256), (257, 320, 2049), (300, 1024, 777), (513, 64, 5000), (1000, 200, 300), (31, 4096, 600), (1, 1024, 20011)]


@pytest.mark.parametrize("t,d,v", SHAPES)
def test_sizes(t, d, v):
    h, w, labels, dloss = make(t, d, v, seed=t + d + v)
    loss, lse = lpq.linear_cross_entropy(h, w, labels)
    check_loss(h, w, labels, loss, lse)
    for fp32 in (False, True):
        dh, dw = lpq.linear_cross_entropy_backward(h, w, labels, lse, dloss, out_fp32=fp32)
        check_grads(h, w, labels, lse, dloss, dh, dw)
    assert lpq.device_status() == 0


@pytest.mark.parametrize("piece", [64, 128, 192, 256, 1024, 4096])
@pytest.mark.parametrize("t", [5, 200, 600])
def test_pieces(piece, t):
    """Any split of the vocabulary, the last piece ragged."""
    h, w, labels, dloss = make(t, 256, 1333, seed=piece)
    _, lse = lpq.linear_cross_entropy(h, w, labels)
    dh, dw = lpq.linear_cross_entropy_backward(h, w, labels, lse, dloss, vocab_piece=piece)
    check_grads(h, w, labels, lse, dloss, dh, dw)


def test_rows_without_target():
    h, w, labels, dloss = make(200, 128, 900, ignore=0.0)
    labels[3], labels[50], labels[199], labels[7] = -1, 900, 1 << 40, -(1 << 62)
    loss, lse = lpq.linear_cross_entropy(h, w, labels)
    check_loss(h, w, labels, loss, lse)
    gone = torch.tensor([3, 50, 199, 7], device="cuda")
    assert not loss[gone].any()
    # whatever such rows hold does not reach the gradients
    dloss[gone] = torch.tensor([float("nan"), float("inf"), -float("inf"), 1e30], device="cuda")
    used = lse.clone()
    used[gone] = float("nan")
    dh, dw = lpq.linear_cross_entropy_backward(h, w, labels, used, dloss)
    assert not dh[gone].any()
    check_grads(h, w, labels, lse, torch.where((labels >= 0) & (labels < 900), dloss, 0.0), dh, dw)
    # no target at all
    labels.fill_(-100)
    loss, lse = lpq.linear_cross_entropy(h, w, labels)
    dh, dw = lpq.linear_cross_entropy_backward(h, w, labels, lse, dloss)
    assert not loss.any() and not dh.any() and not dw.any()


def test_zero_and_uneven_weights():
    """dloss of zero, negative and over many orders of magnitude."""
    h, w, labels, dloss = make(300, 256, 700, ignore=0.0)
    dloss = torch.logspace(-6, 3, 300, device="cuda") * torch.where(torch.arange(300, device="cuda") % 2 == 0, 1.0, -1.0)
    dloss[::7] = 0.0
    _, lse = lpq.linear_cross_entropy(h, w, labels)
    check_grads(h, w, labels, lse, dloss, *lpq.linear_cross_entropy_backward(h, w, labels, lse, dloss))
    zero = torch.zeros_like(dloss)
    dh, dw = lpq.linear_cross_entropy_backward(h, w, labels, lse, zero)
    assert not dh.any() and not dw.any()
    for size in (1e-37, 1e30):
        _, dw = lpq.linear_cross_entropy_backward(h, w, labels, lse, torch.full_like(dloss, size), out_fp32=True)
        _, one = lpq.linear_cross_entropy_backward(h, w, labels, lse, torch.ones_like(dloss), out_fp32=True)
        assert torch.all((dw / size - one).abs() <= 1e-5 * one.abs() + 1e-6)


def test_large_logits():
    """Logits far beyond exp's range."""
    h, w, labels, dloss = make(70, 128, 500, std=30.0)
    loss, lse = lpq.linear_cross_entropy(h, w, labels)
    assert loss.max() > 500
    check_loss(h, w, labels, loss, lse)
    dh, dw = lpq.linear_cross_entropy_backward(h, w, labels, lse, dloss, out_fp32=True)
    assert dh.isfinite().all() and dw.isfinite().all()


def test_special_values():
    h, w, labels, dloss = make(300, 128, 600, ignore=0.0)
    clean, clean_lse = lpq.linear_cross_entropy(h, w, labels)
    h[5, 3] = float("nan")
    h[270, 7] = float("inf")
    loss, lse = lpq.linear_cross_entropy(h, w, labels)
    assert lse[5].isnan() and loss[5].isnan()
    others = torch.ones(300, dtype=torch.bool, device="cuda")
    others[[5, 270]] = False
    assert torch.equal(loss[others], clean[others]) and torch.equal(lse[others], clean_lse[others])
    assert lse[270].item() == float("inf")  # some logits +inf, others -inf
    dh, _ = lpq.linear_cross_entropy_backward(h, w, labels, lse, dloss)
    assert dh[5].isnan().all() and dh[others].isfinite().all()
    # a word no row can produce: its logit is -inf everywhere
    h = h.abs().nan_to_num(1.0, posinf=1.0) + 0.5
    w[17] = -float("inf")
    labels[labels == 17] = 16
    loss, lse = lpq.linear_cross_entropy(h, w, labels)
    rest = torch.cat((w[:17], w[18:]))
    check_loss(h, rest, torch.where(labels > 17, labels - 1, labels), loss, lse)
    # all of them
    w.fill_(-float("inf"))
    _, lse = lpq.linear_cross_entropy(h, w, labels)
    assert torch.all(lse == -float("inf"))


def test_no_rows():
    h, w, labels, dloss = make(0, 64, 100)
    loss, lse = lpq.linear_cross_entropy(h, w, labels)
    assert loss.shape == lse.shape == (0,)
    for fp32 in (False, True):
        dh, dw = lpq.linear_cross_entropy_backward(h, w, labels, lse, dloss, out_fp32=fp32)
        assert dh.shape == (0, 64) and dw.shape == (100, 64) and not dw.any()


def test_strides():
    t, d, v = 130, 192, 400
    big_h, big_w, labels, dloss = make(2 * t, d + 64, 0 + v, seed=5)
    h, w = big_h[::2, 64:], big_w[:, 8:d + 8]
    labels, dloss = labels[:t].contiguous(), dloss[:t].contiguous()
    loss, lse = lpq.linear_cross_entropy(h, w, labels)
    again = lpq.linear_cross_entropy(h.contiguous(), w.contiguous(), labels)
    assert torch.equal(loss, again[0]) and torch.equal(lse, again[1])
    check_loss(h, w, labels, loss, lse)
    check_grads(h, w, labels, lse, dloss, *lpq.linear_cross_entropy_backward(h, w, labels, lse, dloss))


def test_reproducible_and_other_stream():
    h, w, labels, dloss = make(700, 512, 3000)
    loss, lse = lpq.linear_cross_entropy(h, w, labels)
    want = lpq.linear_cross_entropy_backward(h, w, labels, lse, dloss)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for stream in (None, s, s):
        l2, e2 = lpq.linear_cross_entropy(h, w, labels, stream=stream)
        got = lpq.linear_cross_entropy_backward(h, w, labels, lse, dloss, stream=stream)
        junk = [torch.full((1 << 22,), 3.0, device="cuda") for _ in range(4)]
        torch.cuda.synchronize()
        assert torch.equal(l2, loss) and torch.equal(e2, lse)
        for p, q in zip(got, want):
            assert torch.equal(p, q)
        del junk


def test_gradient_against_differences():
    """Central differences of sum(dloss * loss) in 64 bits along random directions."""
    h, w, labels, dloss = make(40, 64, 90, seed=11)
    _, lse = lpq.linear_cross_entropy(h, w, labels)
    dh, dw = lpq.linear_cross_entropy_backward(h, w, labels, lse, dloss, out_fp32=True)
    g = torch.Generator(device="cuda")
    g.manual_seed(2)

    def total(h, w):
        l = h @ w.T
        valid = labels >= 0
        at = l.gather(1, labels.clamp_min(0)[:, None])[:, 0]
        return (torch.where(valid, torch.logsumexp(l, 1) - at, 0.0) * dloss.double()).sum()

    for i, grad in enumerate((dh, dw)):
        step = torch.randn(grad.shape, generator=g, device="cuda", dtype=torch.float64)
        args = [h.double(), w.double()]
        at = lambda s: total(*[a + s * step if j == i else a for j, a in enumerate(args)])
        want = (at(1e-5) - at(-1e-5)) / 2e-5
        # every term of the gradient carries dl's bf16 rounding
        size = dloss.abs().sum().item() * 2 * (args[1 - i].abs().max() * step.abs().mean() * args[0].shape[1]).item()
        assert abs((grad.double() * step).sum() - want) <= 2.0 ** -8 * size


def test_offsets_beyond_32_bits():
    """Vocabulary weights of over 2^31 elements."""
    t, d, v = 12, 4096, (1 << 31) // 4096 + 300
    w = torch.empty(v, d, dtype=BF, device="cuda").normal_(0, 0.02)
    h = torch.empty(t, d, dtype=BF, device="cuda").normal_()
    labels = torch.randint(v - 300, v, (t,), device="cuda")
    dloss = torch.ones(t, device="cuda")
    loss, lse = lpq.linear_cross_entropy(h, w, labels)
    l = torch.cat([h.double() @ c.double().T for c in w.split(65536)], 1)
    off = e(d) * 64 * 1.0
    assert torch.all((lse.double() - torch.logsumexp(l, 1)).abs() <= off + 1e-4)
    assert torch.all((loss.double() - (torch.logsumexp(l, 1) - l.gather(1, labels[:, None])[:, 0])).abs() <= 2 * off + 2e-4)
    dh, dw = lpq.linear_cross_entropy_backward(h, w, labels, lse, dloss)
    dl = (l - lse.double()[:, None]).exp()
    dl[torch.arange(t), labels] -= 1
    for part in (slice(0, 64), slice(v - 300, v)):
        want = dl[:, part].T @ h.double()
        tol = 2.0 ** -8 * (1.1 * dl[:, part].abs().T @ h.double().abs() + want.abs()) + 1e-12
        assert torch.all((dw[part].double() - want).abs() <= tol)
    want = sum(dl[:, i:i + 65536] @ w[i:i + 65536].double() for i in range(0, v, 65536))
    size = sum(dl[:, i:i + 65536].abs() @ w[i:i + 65536].double().abs() for i in range(0, v, 65536))
    assert torch.all((dh.double() - want).abs() <= (2.0 ** -8 + e(v)) * size + 2.0 ** -8 * want.abs())


def test_python_refusals():
    h, w, labels, dloss = make(4, 64, 32)
    _, lse = lpq.linear_cross_entropy(h, w, labels)
    for bad in ((h.float(), w, labels), (h, w[:, :32], labels), (h, w, labels.int()), (h, w, labels[:3]), (h.T, w, labels)):
        with pytest.raises(AssertionError):
            lpq.linear_cross_entropy(*bad)
    for bad, status in (((h[:, :12].contiguous(), w[:, :12].contiguous(), labels), lpq.ERR_SHAPE),
                        ((h[:, 4:12], w[:, 4:12], labels), lpq.ERR_ALIGN), ((h, w[:0], labels), lpq.ERR_SHAPE)):
        with pytest.raises(lpq.LpqError) as err:
            lpq.linear_cross_entropy(*bad)
        assert err.value.status == status
    for piece in (-64, 100):
        with pytest.raises(lpq.LpqError) as err:
            lpq.linear_cross_entropy_backward(h, w, labels, lse, dloss, vocab_piece=piece)
        assert err.value.status == lpq.ERR_SHAPE
