"""Norm and rotation of query and key heads on the GPU against the formulas in 64 bits.

Tolerances: u = 2^-24.  A head's sum of squares takes at most 32 + 5 additions
in any thread and over the lanes: rstd is off by 20 u (half of it, and its own
rounding).  n = x rstd w adds 2 u, cos and sin are off by 4 u (an angle of 2^-26
turns, 1.6 u, and the functions' 2 units), the turn by 3 u: 32 u of |n1| + |n2|.
bf16 outputs add 2^-8 of the value.  An angle far out adds 2^-51 |position
frequency|, which the reference's own product has too."""
import pytest
import torch

from precision_transformer_gemms_gb300 import lpq

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32


def make(t, hq, hk, d, dt, wdt, seed=0, extra=0, pad=0, far=1 << 20):
    """x [t, heads and `extra` columns behind them] in rows `pad` elements longer."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")
    cols = (hq + hk) * d + extra
    x = (r(t, cols + pad) * (0.3 + 3 * r(t, 1).abs())).to(dt)[:, :cols]
    w = [(1 + 0.3 * r(d)).to(wdt) if wdt is not None else None for _ in range(2)]
    pos = torch.randint(-far, far, (t,), generator=g, device="cuda")
    dy = (1e-2 * r(t, (hq + hk) * d)).to(dt)
    return x, w, pos, dy


def turn(v, angle, rot, inter, back=False):
    s, c = angle.sin()[:, None], angle.cos()[:, None]
    s = -s if back else s
    out = v.clone()
    i = (slice(0, rot, 2), slice(1, rot, 2)) if inter else (slice(0, rot // 2), slice(rot // 2, rot))
    a, b = v[..., i[0]], v[..., i[1]]
    out[..., i[0]], out[..., i[1]] = a * c - b * s, b * c + a * s
    return out


def size(v, rot, inter):
    """|v1| + |v2| of every value's pair (|v| of those that are not turned)."""
    v = v.abs()
    out = v.clone()
    i = (slice(0, rot, 2), slice(1, rot, 2)) if inter else (slice(0, rot // 2), slice(rot // 2, rot))
    out[..., i[0]] = out[..., i[1]] = v[..., i[0]] + v[..., i[1]]
    return out


def parts(x, w, hq, hk, d, pos, rot, freqs, eps):
    t = x.shape[0]
    xs = x[:, : (hq + hk) * d].double().reshape(t, hq + hk, d)
    ws = torch.cat([(w[i].double() if w[i] is not None else torch.ones(d, device=x.device, dtype=torch.float64)).expand(n, d)
                    for i, n in ((0, hq), (1, hk))])
    rstd = (xs.square().mean(-1, keepdim=True) + eps).rsqrt()
    f = torch.tensor(freqs, device=x.device, dtype=torch.float64)
    angle = pos.double()[:, None] * f
    slack = 2.0 ** -51 * angle.abs().amax(1) if rot else torch.zeros(t, device=x.device, dtype=torch.float64)
    return xs, ws, rstd, angle, slack[:, None, None]


def custom(rot, base=10000.0):
    return [base ** (-2.0 * i / rot) for i in range(rot // 2)]


def check(x, w, hq, hk, d, pos, y, rot, inter=False, eps=1e-6, freqs=None):
    xs, ws, rstd, angle, slack = parts(x, w, hq, hk, d, pos, rot, custom(rot) if freqs is None else freqs, eps)
    n = xs * rstd * ws
    want = turn(n, angle, rot, inter)
    tol = (32 * U + slack) * size(n, rot, inter) + (2.0 ** -8 if y.dtype == BF else U) * want.abs() + 1e-38
    got = y[:, : (hq + hk) * d].double().view_as(want)
    assert torch.all((got - want).abs() <= tol)


def check_backward(dy, x, w, hq, hk, d, pos, dx, dq, dk, rot, inter=False, eps=1e-6, freqs=None):
    xs, ws, rstd, angle, slack = parts(x, w, hq, hk, d, pos, rot, custom(rot) if freqs is None else freqs, eps)
    dys = dy[:, : (hq + hk) * d].double().reshape(xs.shape)
    g, mag = turn(dys, angle, rot, inter, back=True), size(dys, rot, inter)
    gx = g * ws * xs
    want = rstd * (g * ws - xs * rstd.square() * gx.mean(-1, keepdim=True))
    # g is off by 8 u + the angle's slack of mag; the sums add 40 u of their terms, rstd^3 60 u
    magx = (mag * ws.abs() * xs.abs()).mean(-1, keepdim=True)
    tol = rstd * ((40 * U + slack) * mag * ws.abs() + (120 * U + slack) * xs.abs() * rstd.square() * magx)
    tol = tol + (2.0 ** -8 if dx.dtype == BF else U) * want.abs() + 1e-38
    assert torch.all((dx[:, : (hq + hk) * d].double().view_as(want) - want).abs() <= tol)
    if dq is not None:
        t = xs.shape[0]
        # a warp's run of groups (a 304 * 8th of them, a group is at least a head), then lanes, warps and parts
        k = t * (hq + hk) / 2432 + 5 + 8 + 20 + 16 + 40
        for got, h in ((dq, slice(0, hq)), (dk, slice(hq, hq + hk))):
            assert got.dtype == F32 and got.shape == (d,)
            terms, bound = (g * xs * rstd)[:, h], ((k * U + slack) * mag * xs.abs() * rstd)[:, h]
            assert torch.all((got.double() - terms.sum((0, 1))).abs() <= bound.sum((0, 1)) + 1e-38)


CASES = [  # t, query heads, key heads, head size, turned values, neighbours
    (1, 1, 1, 2, 2, False), (1, 32, 8, 128, 128, False), (3, 5, 1, 64, 64, False), (2, 3, 3, 128, 64, True), (7, 1, 0, 80, 32, False),
    (5, 0, 3, 96, 96, True), (33, 7, 2, 70, 34, False), (9, 6, 2, 72, 36, True), (11, 4, 4, 192, 0, False), (4, 2, 1, 256, 256, False),
    (3, 2, 1, 512, 512, False), (3, 3, 2, 510, 254, True), (2, 2, 2, 300, 300, False), (1025, 3, 1, 16, 16, False), (700, 33, 9, 32, 16, True),
    (3000, 8, 8, 128, 128, False), (6, 3, 1, 26, 0, True), (130, 4, 2, 130, 128, False)]


@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("dt", [BF, F32])
def test_forward_and_backward(case, dt):
    t, hq, hk, d, rot, inter = case
    wdt = {BF: F32, F32: BF}[dt] if d % 3 == 0 else dt
    x, w, pos, dy = make(t, hq, hk, d, dt, wdt, extra=hk * d)
    kw = dict(rotary_dim=rot, interleaved=inter)
    y = lpq.qk_norm_rope(x, hq, hk, d, pos, *w, **kw)
    assert y.shape == (t, (hq + hk) * d) and y.dtype == dt
    check(x, w, hq, hk, d, pos, y, rot, inter)
    dx, dq, dk = lpq.qk_norm_rope_backward(dy, x, hq, hk, d, pos, *w, **kw)
    check_backward(dy, x, w, hq, hk, d, pos, dx, dq, dk, rot, inter)


@pytest.mark.parametrize("case", [  # vectors of 8 bytes; neighbours whose turned part is no multiple of 16
    (50, 5, 3, 80, 40, False), (21, 9, 2, 72, 24, False), (6, 3, 2, 8, 8, False), (5, 2, 1, 24, 8, False), (4, 1, 1, 8, 0, False),
    (400, 7, 2, 104, 52, True), (3, 2, 1, 504, 248, False), (3, 1, 1, 512, 252, True), (9, 8, 4, 128, 52, True), (30, 16, 8, 64, 20, True),
    (2, 3, 1, 488, 484, True), (1500, 4, 4, 40, 24, False)])
@pytest.mark.parametrize("dt", [BF, F32])
def test_smaller_vectors(case, dt):
    test_forward_and_backward(case, dt)


@pytest.mark.parametrize("lead", [4, 12])
def test_rows_that_begin_at_8_bytes(lead):
    t, hq, hk, d = 19, 5, 2, 96
    wide, w, pos, dy = make(t, hq, hk, d, BF, F32, extra=lead, pad=4, seed=8)
    x = wide[:, lead:]
    check(x, w, hq, hk, d, pos, lpq.qk_norm_rope(x, hq, hk, d, pos, *w), d)
    dx, dq, dk = lpq.qk_norm_rope_backward(dy, x, hq, hk, d, pos, *w)
    check_backward(dy, x, w, hq, hk, d, pos, dx, dq, dk, d)


@pytest.mark.parametrize("pad,lead", [(0, 0), (8, 0), (3, 0), (16, 5), (1, 1)])
@pytest.mark.parametrize("dt", [BF, F32])
def test_strides_and_alignment(dt, pad, lead):
    """Rows with gaps, and first columns that no 16 bytes divide."""
    t, hq, hk, d = 21, 3, 2, 64
    wide, w, pos, _ = make(t, hq, hk, d, dt, dt, extra=64 + lead, pad=pad, seed=3)
    x = wide[:, lead:]
    y = lpq.qk_norm_rope(x, hq, hk, d, pos, *w)
    check(x, w, hq, hk, d, pos, y, d)
    dyw = (0.01 * torch.randn(t, (hq + hk) * d + pad, device="cuda")).to(dt)
    dy = dyw[:, : (hq + hk) * d]
    out = torch.full((t, (hq + hk) * d + 7), 5.0, device="cuda", dtype=dt)
    dx, dq, dk = lpq.qk_norm_rope_backward(dy, x, hq, hk, d, pos, *w, out=out)
    check_backward(dy, x, w, hq, hk, d, pos, dx, dq, dk, d)
    assert dx is out and bool((out[:, (hq + hk) * d:] == 5.0).all())


@pytest.mark.parametrize("dt", [BF, F32])
def test_in_place_leaves_the_values_behind_the_keys(dt):
    t, hq, hk, d = 50, 4, 2, 128
    x, w, pos, dy = make(t, hq, hk, d, dt, dt, extra=hk * d)
    want = lpq.qk_norm_rope(x, hq, hk, d, pos, *w)
    mine = x.clone()
    assert lpq.qk_norm_rope(mine, hq, hk, d, pos, *w, out=mine) is mine
    assert torch.equal(mine[:, : (hq + hk) * d], want) and torch.equal(mine[:, (hq + hk) * d:], x[:, (hq + hk) * d:])
    dx, dq, dk = lpq.qk_norm_rope_backward(dy, x, hq, hk, d, pos, *w)
    over = dy.clone()
    got = lpq.qk_norm_rope_backward(over, x, hq, hk, d, pos, *w, out=over)
    assert got[0] is over and torch.equal(over, dx) and torch.equal(got[1], dq) and torch.equal(got[2], dk)


def test_no_weights_and_no_parameter_gradients():
    t, hq, hk, d = 19, 2, 2, 64
    x, _, pos, dy = make(t, hq, hk, d, F32, None)
    check(x, (None, None), hq, hk, d, pos, lpq.qk_norm_rope(x, hq, hk, d, pos), d)
    q = torch.full((d,), 1.5, device="cuda")
    check(x, (q, None), hq, hk, d, pos, lpq.qk_norm_rope(x, hq, hk, d, pos, q_weight=q), d)
    dx, dq, dk = lpq.qk_norm_rope_backward(dy, x, hq, hk, d, pos)
    check_backward(dy, x, (None, None), hq, hk, d, pos, dx, dq, dk, d)
    again, no_q, no_k = lpq.qk_norm_rope_backward(dy, x, hq, hk, d, pos, param_grads=False)
    assert torch.equal(again, dx) and no_q is None and no_k is None


@pytest.mark.parametrize("t", [0, 5])
def test_empty(t):
    d = 64
    x = torch.randn(t, 256, device="cuda")
    pos = torch.zeros(t, device="cuda", dtype=torch.int64)
    hq, hk = (2, 1) if t == 0 else (0, 0)
    y = lpq.qk_norm_rope(x, hq, hk, d, pos)
    assert y.shape == (t, (hq + hk) * d)
    dx, dq, dk = lpq.qk_norm_rope_backward(y, x, hq, hk, d, pos)
    assert dx.numel() == 0 and not dq.any() and not dk.any()
    # heads of one kind alone: the other weight's gradient is 0
    if t:
        _, dq, dk = lpq.qk_norm_rope_backward(torch.randn(t, d, device="cuda"), x, 1, 0, d, pos)
        assert dq.any() and not dk.any()


def test_special_values():
    """A head of zeros gives zeros; NaN and infinities stay in their head."""
    x, w, pos, dy = make(6, 2, 1, 64, F32, F32)
    x = x.contiguous()
    x[0, :64] = 0
    x[1, 70] = float("nan")
    x[2, 5] = float("inf")
    y = lpq.qk_norm_rope(x, 2, 1, 64, pos, *w).view(6, 3, 64)
    assert not y[0, 0].any() and bool(y[1, 1].isnan().all())
    fine = torch.ones(6, 3, dtype=torch.bool, device="cuda")
    fine[1, 1] = fine[2, 0] = False
    assert bool(y[fine].isfinite().all())
    dx, _, _ = lpq.qk_norm_rope_backward(dy, x, 2, 1, 64, pos, *w)
    assert bool(dx.view(6, 3, 64)[fine].isfinite().all())


def test_far_positions_and_own_frequencies():
    hq, hk, d, rot = 2, 1, 64, 32
    x, w, pos, dy = make(40, hq, hk, d, F32, F32, far=1 << 31)
    pos[0], pos[1], pos[2] = 0, (1 << 31) - 1, -(1 << 31)
    check(x, w, hq, hk, d, pos, lpq.qk_norm_rope(x, hq, hk, d, pos, *w, rotary_dim=rot, base=500000.0), rot, freqs=custom(rot, 500000.0))
    freqs = [(-1) ** i * 3.0 / (i + 1) for i in range(rot // 2)]  # beyond a radian, and backwards
    small = pos % 100000
    check(x, w, hq, hk, d, small, lpq.qk_norm_rope(x, hq, hk, d, small, *w, rotary_dim=rot, freqs=freqs), rot, freqs=freqs)
    dx, dq, dk = lpq.qk_norm_rope_backward(dy, x, hq, hk, d, small, *w, rotary_dim=rot, freqs=freqs)
    check_backward(dy, x, w, hq, hk, d, small, dx, dq, dk, rot, freqs=freqs)


def test_gradient_against_differences():
    """<dx, v> + <dw, u> against the 64-bit formula's central difference (step 1e-5:
    its truncation and rounding lie below 1e-8 of the sums of magnitudes, 0.2 u)."""
    t, hq, hk, d, rot = 9, 3, 2, 32, 24
    x, w, pos, dy = make(t, hq, hk, d, F32, F32, far=1000)
    dx, dq, dk = lpq.qk_norm_rope_backward(dy, x, hq, hk, d, pos, *w, rotary_dim=rot)

    def f(step):
        xs, ws, rstd, angle, _ = parts((x.double() + step * v), [w[0].double() + step * vq, w[1].double() + step * vk], hq, hk, d, pos, rot, custom(rot), 1e-6)
        return (turn(xs * rstd * ws, angle, rot, False).reshape(t, -1) * dy.double()).sum()

    for seed in range(3):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        v, vq, vk = (torch.randn(*s, generator=g, device="cuda", dtype=torch.float64) for s in ((t, (hq + hk) * d), (d,), (d,)))
        want = (f(1e-5) - f(-1e-5)) / 2e-5
        terms = [dx.double() * v, dq.double() * vq, dk.double() * vk]
        got, mag = sum(a.sum() for a in terms), sum(a.abs().sum() for a in terms)
        assert abs(got - want) <= 300 * U * mag


def test_same_bits_streams_and_graphs():
    t, hq, hk, d = 515, 4, 2, 128
    x, w, pos, dy = make(t, hq, hk, d, BF, BF)
    y, first = lpq.qk_norm_rope(x, hq, hk, d, pos, *w), lpq.qk_norm_rope_backward(dy, x, hq, hk, d, pos, *w)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y2 = lpq.qk_norm_rope(x, hq, hk, d, pos, *w, stream=s)
    again = lpq.qk_norm_rope_backward(dy, x, hq, hk, d, pos, *w, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(y, y2) and all(torch.equal(a, b) for a, b in zip(first, again))
    graph = torch.cuda.CUDAGraph()
    xs, dys = x.clone(), dy.clone()
    with torch.cuda.graph(graph):
        yg = lpq.qk_norm_rope(xs, hq, hk, d, pos, *w)
        back = lpq.qk_norm_rope_backward(dys, xs, hq, hk, d, pos, *w)
    for scale in (1.0, 2.0):
        xs.copy_(x * scale)
        graph.replay()
        assert torch.equal(yg, lpq.qk_norm_rope(xs, hq, hk, d, pos, *w))
        assert all(torch.equal(a, b) for a, b in zip(back, lpq.qk_norm_rope_backward(dys, xs, hq, hk, d, pos, *w)))


def test_refusals():
    t, hq, hk, d = 5, 2, 1, 64
    x, w, pos, dy = make(t, hq, hk, d, BF, BF)
    good = dict(x=x, q_heads=hq, k_heads=hk, head_dim=d, positions=pos, q_weight=w[0], k_weight=w[1])
    for bad in (dict(x=x.half()), dict(x=x.cpu()), dict(x=x.t()), dict(q_heads=3), dict(positions=pos.int()), dict(positions=pos[:4]), dict(positions=pos.cpu()),
                dict(q_weight=w[0][:32]), dict(q_weight=w[0].float()), dict(k_weight=w[1].cpu()), dict(freqs=[1.0]), dict(out=x.float()), dict(out=x[:4])):
        with pytest.raises(AssertionError):
            lpq.qk_norm_rope(**{**good, **bad})
        with pytest.raises(AssertionError):
            lpq.qk_norm_rope_backward(dy, **{**good, **bad})
    for bad in (dict(rotary_dim=66, head_dim=64), dict(rotary_dim=31), dict(eps=-1.0), dict(freqs=[float("nan")] * 32), dict(x=x[:1].expand(5, -1))):
        with pytest.raises(lpq.LpqError):
            lpq.qk_norm_rope(**{**good, **bad})
    with pytest.raises(AssertionError):
        lpq.qk_norm_rope_backward(dy.float(), **good)
    y = lpq.qk_norm_rope(x, hq, hk, d, pos, rotary_dim=0, freqs=[])
    check(x, (None, None), hq, hk, d, pos, y, 0)
    own = torch.tensor([0.5 ** i for i in range(32)], dtype=torch.float64)  # frequencies of any kind that float() takes
    check(x, w, hq, hk, d, pos % 1000, lpq.qk_norm_rope(**{**good, "positions": pos % 1000, "freqs": own}), d, freqs=own.tolist())
