"""Long sums of the experts' products: many small terms beside a large one that a later
term takes off again.

The tensor core adds 16 products at a time to its sum and drops what lies below the
sum's last bit; 16 of the small terms together are half of that bit.  Sums of 256 columns
that are rounded into the whole keep them.  Tolerance: the large term being L, a rounded
addition is off by 2^-24 L, of which there are columns / 256 in a warp's part and 4 parts
at most; the 16 additions within 256 columns are off by 2^-23 of their sum each (2^-19 of
the small terms; of L only beside the large terms themselves, 2 times 2^-19 L).  The
factors of the hidden value are exact but for 16 u, y rounds to bf16 (2^-8)."""
import pytest
import torch

from precision_transformer_gemms_gb300 import lpq
from test_gpu_moe import values

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
LARGE, SMALL = 2.0 ** 16, 2.0 ** -12


def rows(n, k):
    """n rows of +LARGE, SMALL .., -LARGE, each large one in a block of its own."""
    w = torch.zeros(n, k, device="cuda")
    w[:, 32:k - 32] = SMALL
    w[:, 0], w[:, k - 1] = LARGE / 256, -LARGE / 256  # (times an x of 256)
    return w


def quantized(w):
    return lpq.quantize(w.bfloat16(), lpq.MXFP4, lpq.ROWWISE).row


def bound(k):
    return (k / 256 + 4) * U * LARGE + 2 * 2.0 ** -19 * LARGE + 2.0 ** -19 * k * SMALL


@pytest.mark.parametrize("m", [1, 2, 4, 9])
@pytest.mark.parametrize("d", [32768, 65536])
def test_first_product(m, d):
    f, e = 32, 1
    up = torch.zeros(2, f, d, device="cuda")
    up[0, :, 40] = 2.0  # a gate of 2 in every hidden value
    up[1] = rows(f, d)
    up, down = quantized(up.view(2 * f, d)), quantized(torch.eye(f, device="cuda").repeat(d // f, 1))
    x = torch.ones(m, d, device="cuda")
    x[:, 0] = x[:, -1] = 256.0
    x = x.bfloat16()
    y = lpq.moe(x, up, down, e, torch.zeros(m, 1, device="cuda", dtype=torch.int64), torch.ones(m, 1, device="cuda"))
    gate, lin = (values(up) @ x[0].double()).split(f)
    assert bool((lin == (d - 64) * SMALL).all()) and 4 * bound(d) < (d - 64) * SMALL  # (what is lost is the whole of it)
    silu = torch.nn.functional.silu(gate)
    want = (silu * lin).repeat(d // f)
    assert torch.all((y.double() - want).abs() <= silu.amax() * bound(d) + (16 * U + 2.0 ** -8) * want.abs())


@pytest.mark.parametrize("m", [1, 2, 4, 9])
@pytest.mark.parametrize("f", [32768, 65536])
def test_second_product(m, f):
    d, e = 64, 1
    up = torch.zeros(2, f, d, device="cuda")
    up[0, :, 0] = 1.0  # a gate of 32, whose silu is 32 in FP32
    up[1, :, 1] = 1.0
    up[1, 0, 1], up[1, 0, 32], up[1, -1, 1], up[1, -1, 32] = 0.0, 256.0, 0.0, 256.0
    up, down = quantized(up.view(2 * f, d)), quantized(rows(d, f))
    x = torch.zeros(m, d, device="cuda")
    x[:, 0], x[:, 1], x[:, 32] = 32.0, 2.0 ** -5, 2.0 ** -5
    x = x.bfloat16()
    y = lpq.moe(x, up, down, e, torch.zeros(m, 1, device="cuda", dtype=torch.int64), torch.ones(m, 1, device="cuda"))
    gate, lin = (values(up) @ x[0].double()).split(f)
    want = values(down) @ (torch.nn.functional.silu(gate) * lin)
    assert bool(((want / ((f - 64) * SMALL) - 1).abs() < 1e-6).all()) and 4 * bound(f) < (f - 64) * SMALL
    assert torch.all((y.double() - want).abs() <= bound(f) + (16 * U + 2.0 ** -8) * want.abs())
