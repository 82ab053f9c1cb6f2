"""Hidden values of the experts that nearly cancel in the second product: what is left
of them shows with how many bits they enter it.

Every gate row holds one weight and every up row one or two, so that a gate and an up
value are exact but for the tensor scale's rounding.  Hidden values come in pairs whose
up values differ by some 2^-9 of themselves, and a down row subtracts one pair.
Tolerances, u = 2^-24: h = silu(g) l is off by 16 u of itself (exponential, sum,
quotient, products, two tensor scales), and by 2^-22 of itself and 2^-39 of its vector's
largest as two f16 terms; its product with the down weights by (columns / 16 + 64) 2^-23
of the sum of magnitudes, the sum over the choices by (k + 2) u; y rounds to bf16 (2^-8)."""
import pytest
import torch

from precision_transformer_gemms_gb300 import lpq
from test_gpu_matvec import FORMATS
from test_gpu_moe import values

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def layer(e, f, d, fmt, seed, down_size):
    """d values, of which 0 .. 31 make gates and up values and 32 .. 63 the small differences."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    pick = lambda lo, hi, *s: torch.randint(lo, hi, s, generator=g, device="cuda")
    up = torch.zeros(e, 2, f, d, device="cuda")
    for half in range(2):
        column = pick(0, 32, e, f // 2).repeat_interleave(2, 1)
        up[:, half].scatter_(2, column[..., None], 1.0)
    up[:, 1, 1::2].scatter_(2, pick(32, 64, e, f // 2)[..., None], 2.0 ** -9)
    down = torch.zeros(e, d, f, device="cuda")
    pair = pick(0, f // 2, e, d)[..., None]
    down.scatter_(2, 2 * pair, down_size).scatter_(2, 2 * pair + 1, -down_size)
    quantized = lambda w: lpq.quantize(w.bfloat16(), fmt, lpq.ROWWISE).row
    return quantized(up.view(e * 2 * f, d)), quantized(down.view(e * d, f))


def check(m, d, f, e, k, fmt, down_size=1.0, seed=0):
    up, down = layer(e, f, d, fmt, seed, down_size)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + 1)
    x = torch.randn(m, d, generator=g, device="cuda").bfloat16()
    ids = torch.rand(m, e, generator=g, device="cuda").argsort(1)[:, :k].contiguous()
    probs = torch.rand(m, k, generator=g, device="cuda")
    y = lpq.moe(x, up, down, e, ids, probs)
    wu, wd = values(up).view(e, 2 * f, d), values(down).view(e, d, f)
    loses = False  # one f16 term
    for i, row in enumerate(ids.tolist()):
        want = tol = lost = torch.zeros(d, device="cuda", dtype=torch.float64)
        for j, which in enumerate(row):
            gate, lin = (wu[which] @ x[i].double()).split(f)
            h = torch.nn.functional.silu(gate) * lin
            a, p = wd[which].abs(), probs[i, j].double()
            want = want + p * (wd[which] @ h)
            eh = (16 * U + 2.0 ** -22) * h.abs() + 2.0 ** -39 * h.abs().max()
            tol = tol + p * (a @ eh + ((f / 16 + 64) * 2.0 ** -23 + (k + 2) * U) * (a @ h.abs()))
            scale = 2.0 ** (14 - h.abs().max().log2().floor())
            lost = lost + p * (wd[which] @ ((h * scale).half().double() / scale - h))
        tol = tol + 2.0 ** -8 * want.abs()
        assert torch.all((y[i].double() - want).abs() <= tol), float(((y[i].double() - want).abs() / tol).max())
        loses = loses or bool((lost.abs() > 1.5 * tol).any())
    assert loses or f > 4096


@pytest.mark.parametrize("m,d,f,e,k", [  # columns of an entry: 1, 2, 4 and 8; rows by one warp, and by several
    (1, 64, 64, 2, 1), (1, 256, 2048, 2, 2), (2, 96, 160, 2, 2), (2, 64, 1024, 3, 1), (3, 128, 224, 2, 2), (4, 64, 2080, 8, 3), (16, 96, 96, 2, 1),
    (21, 64, 1056, 3, 2), (8, 1024, 4096, 2, 2)])
@pytest.mark.parametrize("fmt", FORMATS)
def test_differences_of_hidden_values(m, d, f, e, k, fmt):
    check(m, d, f, e, k, fmt, seed=m + f)


@pytest.mark.parametrize("m,k", [(1, 1), (4, 1), (13, 2)])
@pytest.mark.parametrize("size", [2.0 ** 40, 2.0 ** -40])
def test_with_scales_beyond_f16(m, k, size):
    check(m, 64, 288, 2, k, lpq.MXFP4, size)


@pytest.mark.parametrize("m,f", [(1, 65536), (2, 40928), (5, 16384), (9, 8224)])
@pytest.mark.parametrize("fmt", [lpq.NVFP4, lpq.MXFP4])
def test_long_vectors(m, f, fmt):
    check(m, 64, f, 2, 1 + m % 2, fmt)
