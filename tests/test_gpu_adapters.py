"""Products with 4-bit weights and a low-rank adapter for every token, against the
definition in 64 bits.

Tolerance: the products with the weights as in their own test (additions in a row x
2^-23 of sum |x w|).  An inner vector takes at most k / 256 + 16 additions in a row
in FP32, its product with B another rank + 2: (k / 256 + rank + 32) 2^-24 of
scale |B| |A| |x|.  bf16 outputs add 2^-8 of the value."""
import pytest
import torch

from precision_transformer_gemms_gb300 import lpq, synth
from test_gpu_matvec import FORMATS, dequantized, quantized

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def make(n, k, rank, count, m, fmt, layout=lpq.SF_GEMM, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")
    w = quantized(n, k, fmt, layout, seed=seed)
    ad = lpq.Adapters((r(count, rank, k) / k ** 0.5).bfloat16(), r(count, n, rank).bfloat16(), 0.5 + torch.rand(count, generator=g, device="cuda"))
    index = torch.randint(-1, count, (m,), generator=g, device="cuda")
    return w, ad, index, synth.bf16_normal((m, k), 1.0, seed + 7, "cuda", 0.01, 30.0)


def check(x, w, ad, index, y):
    d = torch.from_numpy(dequantized(w)).cuda()
    ts = w.tensor_scale.double().item() if w.fmt != lpq.MXFP4 else 1.0
    want, size = x.double() @ d.T * ts, (x.double().abs() @ d.abs().T) * ts
    tol = (w.cols / 16 + 64) * 2.0 ** -23 * size
    for i, e in enumerate(index.tolist()):
        if 0 <= e < ad.a.shape[0]:
            a, b = ad.a[e].double(), ad.b[e].double()
            scale = ad.scale[e].double() if ad.scale is not None else 1.0
            want[i] += scale * (b @ (a @ x[i].double()))
            tol[i] += (w.cols / 256 + a.shape[0] + 32) * U * scale * (b.abs() @ (a.abs() @ x[i].double().abs()))
    tol = tol + (2.0 ** -8 if y.dtype == torch.bfloat16 else 2.0 ** -22) * want.abs()
    err = (y.double() - want).abs()
    assert torch.all(err <= tol + 1e-38), float((err / (tol + 1e-38)).max())


@pytest.mark.parametrize("n,k,rank,count,m", [
    (16, 32, 8, 1, 1), (48, 64, 8, 3, 2), (384, 512, 8, 3, 1), (80, 160, 40, 2, 3), (1008, 288, 16, 5, 8), (144, 4096, 64, 4, 5), (4096, 128, 16, 7, 9),
    (2000, 1056, 32, 3, 17), (64, 16384, 256, 2, 6), (272, 8224, 24, 6, 40), (12288, 4096, 16, 4, 3), (40000, 2048, 8, 2, 2)])
@pytest.mark.parametrize("fmt", FORMATS)
def test_sizes(n, k, rank, count, m, fmt):
    w, ad, index, x = make(n, k, rank, count, m, fmt, seed=n + k)
    y = lpq.matvec(x, w, adapters=ad, index=index)
    assert y.dtype == torch.bfloat16 and y.shape == (m, n)
    check(x, w, ad, index, y)
    check(x, w, ad, index, lpq.matvec(x, w, out_fp32=True, adapters=ad, index=index))


@pytest.mark.parametrize("fmt", FORMATS)
def test_plain_scales_and_strided_tokens(fmt):
    w, ad, index, x = make(336, 1184, 16, 4, 6, fmt, lpq.SF_PLAIN)
    wide = torch.zeros(6, 1184 + 24, device="cuda", dtype=torch.bfloat16)
    wide[:, :1184] = x
    check(x, w, ad, index, lpq.matvec(wide[:, :1184], w, adapters=ad, index=index))


def test_no_adapter_is_the_plain_product():
    """Tokens whose index lies outside the adapters, whatever it is; the same adapter
    for all; no scale; no adapters at all."""
    w, ad, _, x = make(640, 1024, 16, 3, 5, lpq.NVFP4)
    plain = lpq.matvec(x, w)
    none = torch.tensor([-1, 3, -100, 1 << 40, -(1 << 63)], device="cuda")
    assert torch.equal(lpq.matvec(x, w, adapters=ad, index=none), plain)
    some = torch.tensor([-1, 2, 2, 2, 7], device="cuda")
    y = lpq.matvec(x, w, adapters=ad, index=some)
    check(x, w, ad, some, y)
    assert torch.equal(y[0], plain[0]) and torch.equal(y[4], plain[4])
    unscaled = lpq.Adapters(ad.a, ad.b)
    check(x, w, unscaled, some, lpq.matvec(x, w, adapters=unscaled, index=some))
    empty = lpq.Adapters(ad.a[:0], ad.b[:0])
    assert torch.equal(lpq.matvec(x, w, adapters=empty, index=some), plain)
    assert lpq.matvec(x[:0], w, adapters=ad, index=some[:0]).shape == (0, 640)


def test_an_adapter_of_no_number_stays_with_its_tokens():
    w, ad, _, x = make(320, 512, 8, 3, 4, lpq.NVFP4)
    ad.a[1, 2, 5] = float("nan")
    index = torch.tensor([0, 1, 2, -1], device="cuda")
    y = lpq.matvec(x, w, adapters=ad, index=index)
    assert bool(y[1].isnan().all()) and bool(y[[0, 2, 3]].isfinite().all())


@pytest.mark.parametrize("n,k,m", [(12288, 4096, 8), (4096, 16384, 5), (40000, 1024, 11)])
def test_back_to_back_streams_and_graphs(n, k, m):
    """Calls after one another on one stream, whose kernels overlap; on another stream;
    captured, with inputs and indices changed between replays."""
    w, ad, index, x = make(n, k, 16, 6, m, lpq.NVFP4)
    torch.cuda.synchronize()
    outs = []
    for i in range(6):
        outs.append((x.roll(i, 0), index.roll(2 * i)))
    want = []
    for xi, ii in outs:
        want.append(lpq.matvec(xi, w, adapters=ad, index=ii))
        torch.cuda.synchronize()
    for repeat in range(5):
        got = [lpq.matvec(xi, w, adapters=ad, index=ii) for xi, ii in outs]
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    # inputs written by the kernels just ahead
    for xi, ii in outs:
        fresh, at = torch.zeros_like(x), torch.full_like(index, -1)
        fresh.copy_(xi)
        at.copy_(ii)
        y = lpq.matvec(fresh, w, adapters=ad, index=at)
        fresh.zero_()
        at.fill_(-1)
        assert torch.equal(y, lpq.matvec(xi, w, adapters=ad, index=ii))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y = lpq.matvec(x, w, stream=s, adapters=ad, index=index)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(y, want[0])
    graph, xs, at = torch.cuda.CUDAGraph(), x.clone(), index.clone()
    with torch.cuda.graph(graph):
        h = lpq.matvec(xs, w, adapters=ad, index=at)
        again = lpq.matvec(xs, w, adapters=ad, index=at)
    for (xi, ii), yi in zip(outs, want):
        xs.copy_(xi)
        at.copy_(ii)
        graph.replay()
        assert torch.equal(h, yi) and torch.equal(again, yi)


def test_refusals():
    w, ad, index, x = make(64, 64, 8, 2, 2, lpq.NVFP4)
    for bad in (dict(index=None), dict(index=index[:1]), dict(index=index.int()), dict(index=index.cpu())):
        with pytest.raises(AssertionError):
            lpq.matvec(x, w, adapters=ad, **bad)
    with pytest.raises(AssertionError):
        lpq.matvec(x, w, index=index)
    with pytest.raises(AssertionError):
        lpq.matvec(x, w, adapters=lpq.Adapters(ad.a, torch.zeros(2, 32, 8, device="cuda").bfloat16()), index=index)
    for a, b, s in ((ad.a.float(), ad.b, None), (ad.a[:1], ad.b, None), (ad.a, ad.b[:, :, :4], None), (ad.a.transpose(1, 2), ad.b, None),
                    (ad.a, ad.b, ad.scale[:1]), (ad.a, ad.b, ad.scale.double()), (ad.a.cpu(), ad.b, None)):
        with pytest.raises(AssertionError):
            lpq.Adapters(a, b, s)
    odd = lpq.Adapters(torch.zeros(2, 4, 64, device="cuda").bfloat16(), torch.zeros(2, 64, 4, device="cuda").bfloat16())
    with pytest.raises(lpq.LpqError):
        lpq.matvec(x, w, adapters=odd, index=index)
