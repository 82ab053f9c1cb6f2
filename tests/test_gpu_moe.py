"""A mixture-of-experts layer for a few tokens against its definition in 64 bits.

Tolerances, u = 2^-24.  Router: a logit takes at most d / 32 + 13 additions in a row,
(d / 32 + 13) u of sum |x w| =: e; a probability moves by 2 e of itself, its
exponentials, sum and quotient by 8 u + k u.
Experts: products with the weights are off by (columns / 16 + 64) 2^-23 of sum |x w|
each (the tensor core adds 16 at once).  h = silu(g) l moves by 1.1 |l| of g's error
and |silu(g)| of l's and its own 8 u, and is rounded to 11 bits (2^-11 of itself, 2^-38
of its vector's largest).  y is the products of that with the down weights, weighted
and added in FP32 ((k + 2) u), and rounded to bf16 (2^-8)."""
import functools

import pytest
import torch

from precision_transformer_gemms_gb300 import lpq, synth
from test_gpu_matvec import FORMATS, dequantized

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def weights(e, f, d, fmt, seed=0, std=0.05):
    up = lpq.quantize(synth.bf16_normal((e * 2 * f, d), std, seed, "cuda", 0.01, 10.0), fmt, lpq.ROWWISE).row
    down = lpq.quantize(synth.bf16_normal((e * d, f), std, seed + 1, "cuda", 0.01, 10.0), fmt, lpq.ROWWISE).row
    return up, down


def choices(m, k, e, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    ids = torch.rand(m, e, generator=g, device="cuda").argsort(1)[:, :k].contiguous()
    return ids, torch.rand(m, k, generator=g, device="cuda")


def values(w):
    d = torch.from_numpy(dequantized(w)).cuda()
    return d * (w.tensor_scale.double() if w.fmt != lpq.MXFP4 else 1.0)


def check(x, up, down, e, ids, probs, y):
    d, f, k = up.cols, down.cols, ids.shape[1]
    wu, wd = values(up).view(e, 2 * f, d), values(down).view(e, d, f)
    want, tol = torch.zeros(x.shape, device="cuda", dtype=torch.float64), torch.zeros(x.shape, device="cuda", dtype=torch.float64)
    for i, row in enumerate(ids.tolist()):
        xi = x[i].double()
        for j, which in enumerate(row):
            if not 0 <= which < e:
                continue
            gate, lin = (wu[which] @ xi).split(f)
            eg, el = ((d / 16 + 64) * 2.0 ** -23 * (wu[which].abs() @ xi.abs())).split(f)
            s = torch.nn.functional.silu(gate)
            h = s * lin
            eh = 1.1 * eg * lin.abs() + s.abs() * el + 1.1 * eg * el + (8 * U + 2.0 ** -11) * h.abs() + 2.0 ** -38 * h.abs().max()
            a = wd[which].abs()
            p = probs[i, j].double()
            want[i] += p * (wd[which] @ h)
            tol[i] += p.abs() * (a @ eh + ((f / 16 + 64) * 2.0 ** -23 + (k + 2) * U) * (a @ (h.abs() + eh)))
    tol = tol + 2.0 ** -8 * want.abs() + 1e-38
    err = (y.double() - want).abs()
    assert torch.all(err <= tol), float((err / tol).max())


SHAPES = [  # tokens, hidden, inner, experts, choices
    (1, 32, 32, 1, 1), (1, 512, 384, 8, 2), (2, 96, 64, 3, 2), (3, 160, 160, 5, 4), (5, 2080, 992, 6, 3), (8, 1024, 256, 16, 8), (7, 640, 1216, 4, 1),
    (16, 256, 128, 4, 2), (33, 128, 288, 3, 3), (4, 4096, 64, 4, 2), (2, 64, 4096, 4, 2), (70, 96, 96, 9, 8), (9, 288, 1056, 40, 4)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("fmt", FORMATS)
def test_sizes(shape, fmt):
    m, d, f, e, k = shape
    up, down = weights(e, f, d, fmt, seed=d + f)
    ids, probs = choices(m, k, e, seed=m)
    x = synth.bf16_normal((m, d), 1.0, m, "cuda", 0.01, 30.0)
    y = lpq.moe(x, up, down, e, ids, probs)
    assert y.dtype == torch.bfloat16 and y.shape == (m, d)
    check(x, up, down, e, ids, probs, y)


@functools.lru_cache(maxsize=1)
def many_rows(d, f, fmt):
    return weights(16, f, d, fmt, seed=d)


@pytest.mark.parametrize("d,f,fmt", [(d, f, fmt) for d, f in ((320, 2048), (4000, 96)) for fmt in (lpq.NVFP4, lpq.MXFP4)])
@pytest.mark.parametrize("m,k", [(1, 12), (2, 10), (3, 6), (9, 6)])
def test_more_rows_than_warps(d, f, fmt, m, k):
    """Experts whose rows fill every SM more than once, for all counts of tokens a tile."""
    up, down = many_rows(d, f, fmt)
    ids, probs = choices(m, k, 16, seed=m)
    x = synth.bf16_normal((m, d), 1.0, m, "cuda", 0.01, 30.0)
    check(x, up, down, 16, ids, probs, lpq.moe(x, up, down, 16, ids, probs))


@pytest.mark.parametrize("d,f", [(65536, 32), (32, 65536), (65504, 64), (64, 40928)])
@pytest.mark.parametrize("fmt", [lpq.NVFP4, lpq.MXFP4])
def test_the_longest_rows(d, f, fmt):
    """Vectors of which shared memory holds one or two, for tokens that share an expert."""
    up, down = weights(2, f, d, fmt)
    ids, probs = torch.tensor([[0, 1], [1, 0], [1, -1]], device="cuda"), torch.rand(3, 2, device="cuda")
    x = synth.bf16_normal((3, d), 1.0, 4, "cuda")
    check(x, up, down, 2, ids, probs, lpq.moe(x, up, down, 2, ids, probs))


@pytest.mark.parametrize("fmt", [lpq.NVFP4, lpq.MXFP4])
def test_what_lies_behind_the_last_block_does_not_count(fmt):
    m, d, f, e, k = 4, 288, 96, 3, 2
    up, down = weights(e, f, d, fmt)
    ids, probs = choices(m, k, e)
    x = synth.bf16_normal((m, d), 1.0, 1, "cuda")
    y = lpq.moe(x, up, down, e, ids, probs)
    for w in (up, down):
        blocks, atoms = w.cols // (32 if fmt == lpq.MXFP4 else 16), (w.cols + 255) // 256 * (2 if fmt == lpq.MXFP4 else 4)
        r, b = torch.arange(w.rows, device="cuda")[:, None], torch.arange(blocks, device="cuda")
        held = torch.zeros(w.scales.numel(), device="cuda", dtype=torch.bool)
        held[((r >> 7) * atoms + (b >> 2)) * 512 + (r & 31) * 16 + ((r >> 5) & 3) * 4 + (b & 3)] = True
        flat = w.scales.view(torch.uint8).view(-1)
        flat[~held] = 255 if fmt == lpq.MXFP4 else 127  # no number
    assert torch.equal(lpq.moe(x, up, down, e, ids, probs), y)


@pytest.mark.parametrize("fmts", [(lpq.NVFP4, lpq.MXFP4), (lpq.MXFP4, lpq.NVFP4_2D)])
def test_two_formats_and_strided_tokens(fmts):
    m, d, f, e, k = 6, 480, 352, 5, 2
    up, down = weights(e, f, d, fmts[0])[0], weights(e, f, d, fmts[1])[1]
    ids, probs = choices(m, k, e)
    wide = synth.bf16_normal((m, d + 40), 1.0, 1, "cuda")
    check(wide[:, :d], up, down, e, ids, probs, lpq.moe(wide[:, :d], up, down, e, ids, probs))


def test_every_token_on_one_expert_and_one_expert_twice():
    m, d, f, e = 21, 256, 192, 7
    up, down = weights(e, f, d, lpq.NVFP4)
    x = synth.bf16_normal((m, d), 1.0, 1, "cuda")
    ids = torch.full((m, 2), 6, device="cuda")
    probs = torch.rand(m, 2, device="cuda")
    check(x, up, down, e, ids, probs, lpq.moe(x, up, down, e, ids, probs))


def test_places_without_an_expert():
    m, d, f, e = 6, 256, 192, 4
    up, down = weights(e, f, d, lpq.MXFP4)
    x = synth.bf16_normal((m, d), 1.0, 1, "cuda")
    ids = torch.tensor([[0, 1, 2], [-1, 3, 4], [-1, -1, -1], [1 << 40, 0, -(1 << 63)], [3, 3, -7], [2, 1, 0]], device="cuda")
    probs = torch.rand(m, 3, device="cuda")
    probs[1, 0] = probs[2, 1] = float("nan")  # counts for nothing
    y = lpq.moe(x, up, down, e, ids, probs)
    check(x, up, down, e, ids, torch.nan_to_num(probs), y)
    assert not y[2].any()
    for none in (torch.full((m, 3), -1, device="cuda"), torch.full((m, 3), e, device="cuda")):
        y.fill_(1)
        assert not lpq.moe(x, up, down, e, none, probs).any()
    assert not lpq.moe(x, up, down, e, ids[:, :0].contiguous(), probs[:, :0].contiguous()).any()
    assert lpq.moe(x[:0], up, down, e, ids[:0], probs[:0]).shape == (0, d)


@pytest.mark.parametrize("fmt", FORMATS)
def test_wide_ranges(fmt):
    """Tokens whose values span more than f16 holds, hidden values far beyond it, and a
    token of no number, which stays by itself."""
    m, d, f, e = 5, 512, 256, 4
    up, down = weights(e, f, d, fmt, std=1.0)
    x = synth.bf16_normal((m, d), 1.0, 1, "cuda")
    x[0, ::2] *= 2.0 ** 40
    x[0, 1::2] *= 2.0 ** -40
    x[1] *= 2.0 ** 50
    x[2] *= 2.0 ** -60
    ids, probs = choices(m, 2, e)
    y = lpq.moe(x, up, down, e, ids, probs)
    check(x, up, down, e, ids, probs, y)
    x[3, 7] = float("nan")
    again = lpq.moe(x, up, down, e, ids, probs)
    keep = [0, 1, 2, 4]
    assert bool(again[3].isnan().all()) and torch.equal(again[keep], y[keep])


def test_scales_beyond_f16():
    """MXFP4 groups whose scale f16 cannot hold, with and without codes."""
    m, d, f, e = 3, 256, 128, 2
    up, down = weights(e, f, d, lpq.MXFP4)
    for w in (up, down):
        s = w.scales.view(-1)
        s[::37] = 160
        s[5::41] = 90
    x = synth.bf16_normal((m, d), 2.0 ** -20, 1, "cuda")
    ids, probs = choices(m, 2, e)
    check(x, up, down, e, ids, probs, lpq.moe(x, up, down, e, ids, probs))


def test_same_bits_streams_and_graphs():
    m, d, f, e, k = 8, 1024, 512, 16, 4
    up, down = weights(e, f, d, lpq.NVFP4)
    router = synth.bf16_normal((e, d), 0.03, 5, "cuda")
    cases = [synth.bf16_normal((m, d), 1.0, s, "cuda") for s in range(4)]
    layer = lambda x: lpq.moe(x, up, down, e, *lpq.moe_route(x, router, k))
    want = []
    for x in cases:
        want.append(layer(x))
        torch.cuda.synchronize()
    for _ in range(10):
        got = [layer(x) for x in cases]
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    ids, probs = lpq.moe_route(cases[0], router, k)
    for i in range(m):  # token by token (warps then share rows: other last bits)
        check(cases[0][i:i + 1], up, down, e, ids[i:i + 1], probs[i:i + 1], layer(cases[0][i:i + 1]))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    ids, probs = lpq.moe_route(cases[1], router, k, stream=s)
    y = lpq.moe(cases[1], up, down, e, ids, probs, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(y, want[1])
    graph, x = torch.cuda.CUDAGraph(), cases[0].clone()
    with torch.cuda.graph(graph):
        y, twice = layer(x), layer(x)
    for xi, yi in zip(cases, want):
        x.copy_(xi)
        graph.replay()
        assert torch.equal(y, yi) and torch.equal(twice, yi)


@pytest.mark.parametrize("m,d,e,k", [(1, 8, 1, 1), (1, 512, 8, 2), (2, 4096, 64, 8), (3, 1000, 5, 5), (4, 2880, 32, 4), (7, 7168, 256, 8), (8, 64, 1024, 32), (100, 256, 17, 3),
                                     (5, 72, 9, 2)])
@pytest.mark.parametrize("renormalize", [True, False])
def test_route(m, d, e, k, renormalize):
    g = torch.Generator(device="cuda")
    g.manual_seed(d + e)
    x = torch.randn(m, d, generator=g, device="cuda").bfloat16()
    w = (torch.randn(e, d + 8, generator=g, device="cuda") * 3 / d ** 0.5).bfloat16()[:, :d]
    ids, probs = lpq.moe_route(x, w, k, renormalize=renormalize)
    assert ids.dtype == torch.int64 and probs.dtype == torch.float32 and ids.shape == probs.shape == (m, k)
    logits = x.double() @ w.double().T
    off = ((d / 32 + 13) * U * (x.double().abs() @ w.double().abs().T)).amax(1, keepdim=True)
    best, order = logits.sort(dim=1, descending=True, stable=True)
    clear = torch.ones_like(ids, dtype=torch.bool)
    if e > 1:
        gap = best[:, :-1] - best[:, 1:] > 2 * off
        clear[:, :min(k, e - 1)] &= gap[:, :k]
        clear[:, 1:] &= gap[:, :k - 1]
    assert torch.equal(ids[clear], order[:, :k][clear]) and clear.float().mean() > 0.9
    assert all(len(set(r)) == k for r in ids.tolist())
    chosen = logits.gather(1, ids)
    p = torch.softmax(chosen, 1) if renormalize else torch.softmax(logits, 1).gather(1, ids)
    assert torch.all((probs.double() - p).abs() <= (2 * off + (8 + e) * U) * p + 1e-38)


def test_route_ties_and_special_values():
    """Equal logits go to the lower index: small whole numbers, whose sums are exact."""
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    x = torch.randint(-2, 3, (40, 64), generator=g, device="cuda").bfloat16()
    w = torch.randint(-1, 2, (96, 64), generator=g, device="cuda").bfloat16()
    w[48:] = w[:48]
    ids, _ = lpq.moe_route(x, w, 10)
    assert torch.equal(ids, (x.double() @ w.double().T).sort(dim=1, descending=True, stable=True).indices[:, :10])
    ids, probs = lpq.moe_route(torch.zeros_like(x), w, 3)  # -0 and 0 alike
    assert torch.equal(ids, torch.arange(3, device="cuda").expand(40, 3)) and bool((probs - 1 / 3).abs().max() < 1e-6)
    bad = w.clone()
    bad[0, 0] = float("nan")
    bad[1, 1] = float("inf")
    x[:, :2] = 1
    ids, probs = lpq.moe_route(x, bad, 2)
    assert not (ids == 0).any() and bool((ids[:, 0] == 1).all())
    x[5, 3] = float("nan")
    ids, probs = lpq.moe_route(x, w, 4)
    assert ids[5].tolist() == [0, 1, 2, 3] and bool(probs[5].isnan().all()) and bool(probs[6].isfinite().all())
    assert lpq.moe_route(x[:0], w, 4)[0].shape == (0, 4)


def test_refusals():
    up, down = weights(2, 64, 96, lpq.NVFP4)
    x = synth.bf16_normal((2, 96), 1.0, 1, "cuda")
    ids, probs = choices(2, 2, 2)
    for bad in ((x.float(), up, down, 2, ids, probs), (x, down, down, 2, ids, probs), (x, up, down, 2, ids.int(), probs), (x, up, down, 2, ids, probs.double()),
                (x, up, down, 2, ids[:1], probs), (x, up, down, 2, ids.cpu(), probs)):
        with pytest.raises(AssertionError):
            lpq.moe(*bad)
    with pytest.raises(lpq.LpqError):
        lpq.moe(x, up, down, 3, ids, probs)
    plain = lpq.quantize(synth.bf16_normal((256, 96), 1.0, 1, "cuda"), lpq.NVFP4, lpq.ROWWISE, sf_layout=lpq.SF_PLAIN).row
    with pytest.raises(lpq.LpqError):
        lpq.moe(x, plain, down, 2, ids, probs)
    with pytest.raises(lpq.LpqError):
        lpq.moe_route(x, torch.zeros(3, 96, device="cuda").bfloat16(), 4)
