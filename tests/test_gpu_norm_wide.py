"""Layer norm of rows beyond 16384 columns: whole vectors and single elements,
strides, optional parameters, more rows than CTAs, the amax."""
import pytest
import torch

from precision_transformer_gemms_gb300 import lpq
from test_gpu_norm import check_backward, check_forward, make

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("rows,cols", [(1, 16385), (2, 16388), (3, 16392), (7, 20000), (5, 32767), (700, 16392), (400, 16390), (2, 262144)])
@pytest.mark.parametrize("dt,wdt", [(BF, BF), (BF, F32), (F32, F32), (F32, BF)])
def test_forward_and_backward(rows, cols, dt, wdt):
    x, w, b, dy = make(rows, cols, dt, wdt, seed=cols)
    amax = torch.full((1,), -1.0, device="cuda")
    y, mean, rstd = lpq.layer_norm(x, w, b, amax=amax)
    check_forward(x, w, b, 1e-5, y, mean, rstd)
    assert amax.item() == y.float().abs().max().item()
    check_backward(dy, x, w, mean, rstd, *lpq.layer_norm_backward(dy, x, mean, rstd, w))


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("cols,pad,start", [(16640, 8, 0), (16640, 3, 0), (16640, 64, 1), (17000, 40, 8)])
def test_strides_and_alignment(dt, cols, pad, start):
    big, w, b, dbig = make(9, cols + pad, dt, dt)
    x, dy = big[:, start:start + cols], dbig[:, start:start + cols]
    w, b = w[start:start + cols], b[start:start + cols]
    out = torch.full((9, cols + pad), 7.0, dtype=dt, device="cuda")
    y, mean, rstd = lpq.layer_norm(x, w, b, out=out[:, start:start + cols])
    check_forward(x, w, b, 1e-5, y, mean, rstd)
    assert torch.all(out[:, :start] == 7) and torch.all(out[:, start + cols:] == 7)
    check_backward(dy, x, w, mean, rstd, *lpq.layer_norm_backward(dy, x, mean, rstd, w))


@pytest.mark.parametrize("cols", [16392, 16393])
@pytest.mark.parametrize("w_on,b_on", [(False, False), (True, False), (False, True)])
def test_optional_parameters(w_on, b_on, cols):
    x, w, b, dy = make(5, cols, BF, BF)
    w, b = (w if w_on else None), (b if b_on else None)
    y, mean, rstd = lpq.layer_norm(x, w, b)
    check_forward(x, w, b, 1e-5, y, mean, rstd)
    check_backward(dy, x, w, mean, rstd, *lpq.layer_norm_backward(dy, x, mean, rstd, w))


def test_special_rows():
    x, w, b, dy = make(6, 16400, BF, BF)
    x[1], x[2, 5], x[3, 16399] = 3.0, float("nan"), float("inf")
    y, mean, rstd = lpq.layer_norm(x, w, b)
    keep = [0, 1, 4, 5]
    check_forward(x[keep], w, b, 1e-5, y[keep], mean[keep], rstd[keep])
    assert torch.equal(y[1], b) and y[2].isnan().all() and y[3].isnan().all()
    dx, dw, db = lpq.layer_norm_backward(dy, x, mean, rstd, w)
    check_backward(dy[keep], x[keep], w, mean[keep], rstd[keep], dx[keep], None, None)
    assert dx[2].isnan().all() and dw.isnan().all() and not db.isnan().any()
