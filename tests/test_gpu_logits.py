"""Penalties, biases and masks on logits against the definition in 64 bits.

Tolerance: u = 2^-24 of every intermediate's size: the division or product, the
product f c, two differences and the bias (whose own sum has at most n more
additions): 5 u (|l| + |f c| + |p|) + (n + 1) u sum|b|; bf16 adds 2^-8 of the value."""
import math

import pytest
import torch

from precision_transformer_gemms_gb300 import lpq
from precision_transformer_gemms_gb300.head import LanguageHead

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32


def make(t, v, n, dt, seed=0, biases=5, pad=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    r = lambda *s: torch.rand(*s, generator=g, device="cuda")
    logits = (8 * (r(t, v + pad) - 0.5)).to(dt)[:, :v]
    history = (r(t, n) ** 3 * v).long().clamp_max(v - 1)
    lengths = (r(t) * (n + 1)).long().clamp_max(n)
    prompt = (r(t) * (lengths + 1)).long()
    if n:
        lengths[-1] = n
        history[0, ::5] = -1  # padding counts for nothing
        history[-1, ::7] = v
    offsets = torch.zeros(t + 1, device="cuda", dtype=torch.int64)
    offsets[1:] = (r(t) * (biases + 1)).long().cumsum(0)
    count = int(offsets[-1])
    words = (r(count) * v).long().clamp_max(v - 1)
    values = 3 * torch.randn(count, generator=g, device="cuda")
    allowed = torch.randint(-(1 << 31), 1 << 31, (t, (v + 31) // 32), generator=g, device="cuda").int()
    return logits, dict(history=history, lengths=lengths, prompt=prompt, repetition=1 + r(t), frequency=r(t), presence=r(t),
                        bias=(offsets, words, values), allowed=allowed)


def check(logits, c, got):
    (t, v), inf = logits.shape, math.inf
    x = logits.double().clone()
    slack = torch.zeros_like(x)
    h, lengths = c.get("history"), c.get("lengths")
    one = torch.ones(t, device="cuda", dtype=torch.float64)
    rep, freq, pres = (c[k].double() if c.get(k) is not None else z for k, z in (("repetition", one), ("frequency", 0 * one), ("presence", 0 * one)))
    for i in range(t):
        if h is not None:
            n = max(0, min(int(lengths[i]), h.shape[1]))
            p = max(0, min(int(c["prompt"][i]), n)) if c.get("prompt") is not None else 0
            for words, answer in ((h[i, :n], False), (h[i, p:n], True)):
                words = words[(words >= 0) & (words < v)]
                ids, times = torch.unique(words, return_counts=True)
                old = x[i, ids]
                if answer:
                    x[i, ids] -= freq[i] * times + pres[i]
                    slack[i, ids] += 5 * U * (freq[i] * times + pres[i]).abs()
                else:
                    x[i, ids] = torch.where(old > 0, old / rep[i], old * rep[i])
                    slack[i, ids] += 5 * U * x[i, ids].abs()
        if c.get("bias") is not None:
            offsets, words, values = c["bias"]
            a, z = max(0, int(offsets[i])), min(int(offsets[i + 1]), words.numel())
            for w, b in zip(words[a:z].tolist(), values[a:z].tolist()):
                if 0 <= w < v:
                    x[i, w] += b
                    slack[i, w] += (z - a + 1) * U * abs(b) + 5 * U * abs(logits[i, w].item())
        if c.get("allowed") is not None:
            bits = (c["allowed"][i][:, None] >> torch.arange(32, device="cuda", dtype=torch.int32)) & 1
            x[i, bits.flatten()[:v] == 0] = -inf
    fine = x.isfinite()
    assert torch.equal(got[~fine & ~x.isnan()].double(), x[~fine & ~x.isnan()]) and torch.equal(got.isnan(), x.isnan())
    tol = slack + (2.0 ** -8 if got.dtype == BF else U) * x.abs()
    assert torch.all((got.double() - x).abs()[fine] <= tol[fine])


@pytest.mark.parametrize("t,v,n", [(1, 1, 1), (1, 31, 4), (2, 33, 0), (3, 1000, 50), (5, 4097, 700), (1, 32000, 3000), (9, 131073, 20), (64, 50257, 300)])
@pytest.mark.parametrize("dt", [BF, F32])
def test_all_controls(t, v, n, dt):
    logits, c = make(t, v, n, dt, seed=t + v)
    check(logits, c, lpq.adjust_logits(logits, **c))


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("drop", ["history", "bias", "allowed", "prompt", "repetition", "frequency", "presence", "but_bias", "but_allowed", "all"])
def test_any_control_may_be_left_out(drop, dt):
    logits, c = make(4, 999, 60, dt, seed=2)
    groups = {"history": ("history", "lengths", "prompt", "repetition", "frequency", "presence")}
    keep = {"but_bias": ("bias",), "but_allowed": ("allowed",), "all": ()}.get(drop)
    c = {k: v for k, v in c.items() if (k in keep if keep is not None else k not in groups.get(drop, (drop,)))}
    y = lpq.adjust_logits(logits, **c)
    check(logits, c, y)
    if drop == "all":
        assert torch.equal(y, logits)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("pad,lead,opad,olead", [(0, 0, 0, 0), (1, 0, 1, 0), (3, 2, 3, 2), (5, 1, 0, 0), (0, 3, 8, 3), (16, 8, 0, 0), (2, 0, 1, 1)])
def test_strides_and_alignment(dt, pad, lead, opad, olead):
    t, v = 5, 4500
    logits, c = make(t, v + lead, 40, dt, seed=4, pad=pad)
    logits = logits[:, lead:]
    c["allowed"] = c["allowed"][:, : (v + 31) // 32]
    out = torch.full((t, olead + v + opad), 7.0, device="cuda", dtype=dt)
    y = lpq.adjust_logits(logits, **c, out=out[:, olead:olead + v])
    check(logits, c, y)
    assert bool((out[:, :olead] == 7).all()) and bool((out[:, olead + v:] == 7).all())


@pytest.mark.parametrize("t", [2, 400])
def test_in_place_and_streams(t):
    logits, c = make(t, 10001, 100, F32, seed=5)
    want = lpq.adjust_logits(logits, **c)
    mine = logits.clone()
    assert lpq.adjust_logits(mine, **c, out=mine) is mine and torch.equal(mine, want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = lpq.adjust_logits(logits, **c, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(other, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = lpq.adjust_logits(logits, **c)
    logits.mul_(-1)
    c["lengths"].clamp_(max=3)
    graph.replay()
    check(logits, c, got) if t < 10 else None
    assert torch.equal(got, lpq.adjust_logits(logits, **c))


def test_special_values_and_bad_entries():
    v = 2000
    logits, c = make(4, v, 30, F32, seed=6)
    logits = logits.contiguous()
    logits[0, :9] = math.nan
    logits[1, :9] = math.inf
    logits[2, :9] = -math.inf
    c["allowed"][0, :5] = 0
    c["allowed"][3] = 0  # a row that may say nothing
    c["lengths"][0], c["lengths"][1] = -5, 10 ** 12  # taken within the history
    c["history"][1, 3], c["history"][1, 4] = -(1 << 63), (1 << 63) - 1
    y = lpq.adjust_logits(logits, **c)
    check(logits, c, y)
    assert bool((y[3] == -math.inf).all())
    offsets, words, values = c["bias"]
    offsets, words = offsets.clone(), words.clone()
    offsets[0], offsets[-1] = -7, 10 ** 9  # taken within the list
    words[::2] = -3
    c["bias"] = offsets, words, values
    check(logits, c, lpq.adjust_logits(logits, **c))


def test_repetition_of_any_size():
    """Divisors without a reciprocal among the normal numbers, too: a correctly rounded
    quotient or product is off by half a step, or half of 2^-149 below 2^-126."""
    r = torch.tensor([1e-40, 2.0 ** -126, 2.0 ** -127, 3e38, 2.0 ** 126, math.inf, 0.0, -1.5], device="cuda")
    v = 600
    g = torch.Generator(device="cuda")
    g.manual_seed(11)
    logits = 1e-3 * torch.randn(len(r), v, generator=g, device="cuda")
    words = torch.arange(v, device="cuda").repeat(len(r), 1)
    got = lpq.adjust_logits(logits, words, torch.full((len(r),), v, device="cuda"), repetition=r).double()
    x, d = logits.double(), r.double()[:, None]
    want = torch.where(x > 0, x / d, x * d)
    fine = want.isfinite()
    assert torch.equal(got[~fine], want[~fine])
    assert torch.all((got - want).abs()[fine] <= (2 * U * want.abs() + 2.0 ** -149)[fine])


def test_biases_of_one_word_add_in_order():
    logits = torch.zeros(2, 700, device="cuda")
    values = torch.tensor([1e8, 1.0, -1e8, 5.0, 3.0] * 20, device="cuda")
    words = torch.tensor([5, 5, 5, 699, 5] * 20, device="cuda")
    y = lpq.adjust_logits(logits, bias=(torch.tensor([0, 100, 100], device="cuda"), words, values))
    total = torch.zeros((), dtype=F32)
    for w, b in zip(words.tolist(), values.cpu()):
        total = total + b if w == 5 else total
    assert y[0, 5].item() == total.item() and y[0, 699].item() == 100.0 and not y[1].any()


def test_empty():
    for t, v in ((0, 100), (3, 0), (0, 0)):
        c = dict(history=torch.zeros(t, 0, device="cuda", dtype=torch.int64), lengths=torch.zeros(t, device="cuda", dtype=torch.int64),
                 repetition=torch.ones(t, device="cuda"))
        assert lpq.adjust_logits(torch.empty(t, v, device="cuda"), **c).shape == (t, v)


def test_the_head_applies_them_in_place():
    g = torch.Generator(device="cuda")
    g.manual_seed(0)
    d, v, t = 256, 1104, 3
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")
    head = LanguageHead((1 + 0.1 * r(d)).bfloat16(), (0.1 * r(d)).bfloat16(), (0.05 * r(v, d)).bfloat16()).freeze()
    x = r(t, d).bfloat16()
    _, c = make(t, v, 40, F32)
    plain = head.logits(x)
    want = lpq.adjust_logits(plain, **c)
    assert torch.equal(head.logits(x, controls=c), want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = head.logits(x, stream=s, controls=c)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(other, want)
