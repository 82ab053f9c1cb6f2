"""Rotation at positions up to 2^50 with frequencies small and large, of both signs,
against angles from exact arithmetic.  The tolerance of a turned pair: u = 2^-24, 32 u of
|n1| + |n2| for the statistics, the products and an angle rounded to 2^-26 turns, and
2^-52 |position frequency| of its own pair's; u of the value (FP32)."""
import math
from fractions import Fraction

import pytest
import torch

from precision_transformer_gemms_gb300 import lpq
from test_turns import PI

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
FREQS = [1.0, -1.0, 1e-3, -1e-3, 500000.0 ** (-126 / 128), -500000.0 ** (-126 / 128), 2.0 ** -30, -2.0 ** -30]
POSITIONS = [s * p for p in [0, 1, 511, 1 << 20, (1 << 31) + 5, 1 << 36, 1 << 40, (1 << 45) + 12345, (1 << 50) - 1, 1 << 50] for s in (1, -1)]


def exact_angle(position, frequency):
    turns = Fraction(position) * Fraction(frequency) / (2 * PI) % 1
    return float((turns if turns < Fraction(1, 2) else turns - 1) * 2 * PI)


def turned(v, angle, interleaved, sign):
    a, b = (v[..., 0::2], v[..., 1::2]) if interleaved else v.chunk(2, -1)
    c, s = angle.cos()[:, None], sign * angle.sin()[:, None]
    pair, size = (a * c - b * s, b * c + a * s), a.abs() + b.abs()
    join = (lambda p, q: torch.stack((p, q), -1).flatten(-2)) if interleaved else (lambda p, q: torch.cat((p, q), -1))
    return join(*pair), join(size, size), join


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("pad", [0, 1])  # in vectors, and value by value
def test_far_positions(interleaved, pad):
    t, d, heads = len(POSITIONS), 2 * len(FREQS), 3
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")
    x, dy = r(t, heads * d + pad)[:, :heads * d], r(t, heads * d)
    positions = torch.tensor(POSITIONS, device="cuda")
    angle = torch.tensor([[exact_angle(p, f) for f in FREQS] for p in POSITIONS], device="cuda", dtype=torch.float64)
    slack = torch.tensor([[2.0 ** -52 * abs(p * f) for f in FREQS] for p in POSITIONS], device="cuda", dtype=torch.float64)[:, None]
    kw = dict(freqs=FREQS, interleaved=interleaved)
    y = lpq.qk_norm_rope(x, 2, 1, d, positions, **kw).double().view(t, heads, d)
    xs = x.double().reshape(t, heads, d)
    rstd = (xs.square().mean(-1, keepdim=True) + 1e-6).rsqrt()
    want, size, join = turned(xs * rstd, angle, interleaved, 1)
    pairs = join(slack, slack)
    assert torch.all((y - want).abs() <= (32 * U + pairs) * size + U * want.abs())

    dx = lpq.qk_norm_rope_backward(dy, x, 2, 1, d, positions, **kw)[0].double().view(t, heads, d)
    turn_back, size, _ = turned(dy.double().view(t, heads, d), angle, interleaved, -1)
    want = rstd * (turn_back - xs * rstd.square() * (turn_back * xs).mean(-1, keepdim=True))
    # as in the test of all sizes: g is off by 8 u + its angle's of its pair, the sums by 40 u, rstd^3 by 60 u
    dot = ((120 * U + pairs) * size * xs.abs()).mean(-1, keepdim=True)
    assert torch.all((dx - want).abs() <= rstd * ((40 * U + pairs) * size + xs.abs() * rstd.square() * dot) + U * want.abs())
    assert math.isclose(exact_angle(1, 1.0), 1.0)
