"""Rows of one value: the mean is that value, the variance 0 and y the bias, exactly.

A value c of b significant bits times any count up to 2^(24 - b) is an FP32
number, so every partial sum is exact and sum / n is c."""
import pytest
import torch

from precision_transformer_gemms_gb300 import lpq

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cols", [1, 3, 7, 24, 100, 257, 520, 1000, 1023, 1544, 2047, 3080, 4095, 5000, 8191, 12345, 16383, 16400, 33333])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_constant_rows(cols, dt):
    c = torch.tensor([0.0, 1.0, -3.0, 1000.0, -1992.0, 99840.0, 6.9e8, 1.17e-5, 0.1], device="cuda").bfloat16().to(dt)
    x = c[:, None].expand(-1, cols).contiguous()
    g = torch.Generator(device="cuda")
    g.manual_seed(cols)
    weight, bias = (torch.randn(cols, generator=g, device="cuda").to(dt) for _ in range(2))
    y, mean, rstd = lpq.layer_norm(x, weight, bias, eps=1e-5)
    assert torch.equal(mean, c.float())
    assert torch.equal(y, bias.expand_as(x))
    assert torch.allclose(rstd, torch.full_like(rstd, 1e-5).rsqrt(), rtol=2.0 ** -22, atol=0)
