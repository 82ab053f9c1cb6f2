"""Layer norm and its backward pass on the GPU against the formulas in 64 bits.

Tolerances: u = 2^-24 is FP32's rounding unit.  A row's sums run over at most
n / 256 + 24 consecutive additions in any of the kernels, so a mean of values
up to A is off by at most k u A with k = n / 256 + 32 (which covers the few
roundings around the sums); bf16 outputs add half a unit in the last place,
2^-8 of the value."""
import pytest
import torch

from precision_transformer_gemms_gb300 import lpq

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32


def make(rows, cols, dt, wdt, seed=0, offset=0.0, affine=True):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")
    x = (r(rows, cols) * 2 + r(rows, 1) + offset).to(dt)
    w = (1 + 0.2 * r(cols)).to(wdt) if affine else None
    b = (0.3 * r(cols)).to(wdt) if affine else None
    return x, w, b, (1e-2 * r(rows, cols)).to(dt)


def ref_forward(x, w, b, eps):
    x = x.double()
    mean = x.mean(1)
    c = x - mean[:, None]
    rstd = (c.square().mean(1) + eps).rsqrt()
    y = c * rstd[:, None]
    if w is not None:
        y = y * w.double()
    if b is not None:
        y = y + b.double()
    return y, mean, rstd


def check_forward(x, w, b, eps, y, mean, rstd):
    y64, m64, r64 = ref_forward(x, w, b, eps)
    n = x.shape[1]
    k = n / 256 + 32
    top = x.double().abs().amax(1)
    off = k * U * top  # of the mean and of every centred value
    assert torch.all((mean.double() - m64).abs() <= off)
    rel = 2 * k * U + (off * r64) ** 2
    assert torch.all((rstd.double() - r64).abs() <= rel * r64)
    aw = w.double().abs() if w is not None else torch.ones(n, device=x.device, dtype=torch.float64)
    ab = b.double().abs() if b is not None else torch.zeros(n, device=x.device, dtype=torch.float64)
    xh = ((x.double() - m64[:, None]) * r64[:, None]).abs()
    tol = (2 * off * r64)[:, None] * aw + (rel[:, None] + 4 * U) * xh * aw + 2 * U * ab
    tol = tol + (2.0 ** -8 if y.dtype == BF else U) * y64.abs() + 1e-38
    assert torch.all((y.double() - y64).abs() <= tol)


def check_backward(dy, x, w, mean, rstd, dx, dw, db):
    n, rows = x.shape[1], x.shape[0]
    k = n / 256 + 32
    m, r, d = mean.double()[:, None], rstd.double()[:, None], dy.double()
    xh = (x.double() - m) * r
    xe = 4 * U * (x.double().abs() + m.abs()) * r  # xhat's own rounding
    g = d * (w.double() if w is not None else 1.0)
    dx64 = r * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
    size = g.abs() + g.abs().mean(1, keepdim=True) + xh.abs() * (g * xh).abs().mean(1, keepdim=True)
    fuzz = xe * (g * xh).abs().mean(1, keepdim=True) + xh.abs() * (g.abs() * xe).mean(1, keepdim=True)
    tol = 2 * r * (k * U * size + fuzz) + (2.0 ** -8 if dx.dtype == BF else U) * dx64.abs() + 1e-38
    assert torch.all((dx.double() - dx64).abs() <= tol)
    if dw is not None:
        # rows / parts additions inside a part (a part is 1 / 304 of the rows, at least one), then the parts
        kr = (rows / 256 + 304 + 64) * U
        assert dw.dtype == F32 and db.dtype == F32
        assert torch.all((dw.double() - (d * xh).sum(0)).abs() <= (kr * (d * xh).abs() + d.abs() * xe).sum(0) + 1e-38)
        assert torch.all((db.double() - d.sum(0)).abs() <= kr * d.abs().sum(0) + 1e-38)


SHAPES = [(1, 1), (1, 8), (3, 7), (5, 64), (2, 100), (33, 256), (17, 1000), (64, 1023), (9, 1024), (300, 520), (40, 2048),
          (31, 4096), (700, 768), (7, 8192), (5, 12345), (3, 16384), (2, 40000)]


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("dt,wdt", [(BF, BF), (BF, F32), (F32, F32), (F32, BF)])
def test_forward_and_backward(rows, cols, dt, wdt):
    x, w, b, dy = make(rows, cols, dt, wdt, seed=rows + cols)
    y, mean, rstd = lpq.layer_norm(x, w, b, eps=1e-5)
    assert y.dtype == dt and mean.dtype == rstd.dtype == F32
    check_forward(x, w, b, 1e-5, y, mean, rstd)
    check_backward(dy, x, w, mean, rstd, *lpq.layer_norm_backward(dy, x, mean, rstd, w))


@pytest.mark.parametrize("w_on,b_on", [(False, False), (True, False), (False, True)])
@pytest.mark.parametrize("cols", [96, 4096, 4097])
def test_optional_parameters(w_on, b_on, cols):
    x, w, b, dy = make(37, cols, BF, BF)
    w, b = (w if w_on else None), (b if b_on else None)
    y, mean, rstd = lpq.layer_norm(x, w, b)
    check_forward(x, w, b, 1e-5, y, mean, rstd)
    check_backward(dy, x, w, mean, rstd, *lpq.layer_norm_backward(dy, x, mean, rstd, w))
    dx, dw, db = lpq.layer_norm_backward(dy, x, mean, rstd, w, param_grads=False)
    assert dw is None and db is None
    check_backward(dy, x, w, mean, rstd, dx, None, None)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("cols,pad,start", [(1024, 8, 0), (1024, 3, 0), (1024, 64, 1), (520, 40, 8), (4096, 4096, 0), (768, 5, 2)])
def test_strides_and_alignment(dt, cols, pad, start):
    """Rows apart by more than their length, and rows that start anywhere."""
    rows = 45
    big, w, b, dbig = make(rows, cols + pad, dt, BF)
    x, dy = big[:, start:start + cols], dbig[:, start:start + cols]
    w, b = w[start:start + cols], b[start:start + cols]
    out = torch.full((rows, cols + pad), 7.0, dtype=dt, device="cuda")
    y, mean, rstd = lpq.layer_norm(x, w, b, out=out[:, start:start + cols])
    check_forward(x, w, b, 1e-5, y, mean, rstd)
    assert torch.all(out[:, :start] == 7) and torch.all(out[:, start + cols:] == 7)
    check_backward(dy, x, w, mean, rstd, *lpq.layer_norm_backward(dy, x, mean, rstd, w))


def test_large_offset_keeps_digits():
    """A row far from zero: the variance comes from the centred values."""
    x, w, b, _ = make(20, 4096, F32, F32, offset=1000.0)
    y, mean, rstd = lpq.layer_norm(x, w, b)
    check_forward(x, w, b, 1e-5, y, mean, rstd)


def test_constant_and_special_rows():
    x, w, b, dy = make(8, 1024, BF, BF)
    x[1] = 3.0                      # no variance: y = bias
    x[2] = 0.0
    x[4, 5] = float("nan")
    x[5, 6] = float("inf")
    x[6] = 3e38                     # its sum leaves the FP32 range
    amax = torch.full((1,), -1.0, device="cuda")
    y, mean, rstd = lpq.layer_norm(x, w, b, amax=amax)
    keep = [0, 1, 2, 3, 7]
    check_forward(x[keep], w, b, 1e-5, y[keep], mean[keep], rstd[keep])
    assert torch.equal(y[1], b) and torch.equal(y[2], b)
    assert y[4].isnan().all() and y[5].isnan().all()
    assert amax.item() == y[[0, 1, 2, 3, 6, 7]].float().nan_to_num(0.0, float("inf")).abs().max().item()
    dx, dw, db = lpq.layer_norm_backward(dy, x, mean, rstd, w)
    check_backward(dy[keep], x[keep], w, mean[keep], rstd[keep], dx[keep], None, None)
    assert dx[4].isnan().all() and dw.isnan().all() and not db.isnan().any()


@pytest.mark.parametrize("rows,cols,dt", [(1, 16, BF), (700, 4096, BF), (65, 777, F32), (300, 256, BF)])
def test_amax_is_the_quantizers(rows, cols, dt):
    x, w, b, _ = make(rows, cols, dt, BF)
    amax = torch.full((1,), 1e30, device="cuda")
    y, _, _ = lpq.layer_norm(x, w, b, amax=amax)
    assert amax.item() == y.float().abs().max().item()
    if dt == BF and cols % 16 == 0:
        assert amax.item() == lpq.amax(y)[0].item()


def test_norm_feeds_the_quantizer():
    """quantize with the norm's amax gives exactly what quantize computes alone."""
    x, w, b, _ = make(256, 512, BF, BF)
    ref = lpq.alloc(lpq.NVFP4, 256, 512, lpq.ROWWISE)
    y, _, _ = lpq.layer_norm(x, w, b, amax=ref.row.amax)
    lpq.quantize(y, lpq.NVFP4, lpq.ROWWISE | lpq.GIVEN_AMAX, out=ref)
    alone = lpq.quantize(y, lpq.NVFP4, lpq.ROWWISE)
    assert torch.equal(ref.row.codes, alone.row.codes) and torch.equal(ref.row.scales, alone.row.scales)


@pytest.mark.parametrize("cols", [64, 1000, 1023, 4096])
def test_no_rows(cols):
    x, w, b, dy = make(0, cols, BF, BF)
    amax = torch.full((1,), 5.0, device="cuda")
    y, mean, rstd = lpq.layer_norm(x, w, b, amax=amax)
    assert y.shape == (0, cols) and amax.item() == 0
    dx, dw, db = lpq.layer_norm_backward(dy, x, mean, rstd, w)
    assert dx.shape == (0, cols) and not dw.any() and not db.any()


def test_backward_is_reproducible():
    x, w, b, dy = make(3001, 2048, BF, BF)
    y, mean, rstd = lpq.layer_norm(x, w, b)
    first = lpq.layer_norm_backward(dy, x, mean, rstd, w)
    for _ in range(3):
        for p, q in zip(first, lpq.layer_norm_backward(dy, x, mean, rstd, w)):
            assert torch.equal(p, q)


@pytest.mark.parametrize("cols", [48, 1021, 2048])
def test_gradient_against_differences(cols):
    """Central differences of sum(dy * norm(x)) in 64 bits along random directions."""
    x, w, b, dy = make(6, cols, F32, F32, seed=3)
    y, mean, rstd = lpq.layer_norm(x, w, b)
    dx, dw, db = lpq.layer_norm_backward(dy, x, mean, rstd, w)
    f = lambda x, w, b: (ref_forward(x, w, b, 1e-5)[0] * dy.double()).sum()
    g = torch.Generator(device="cuda")
    g.manual_seed(9)
    for i, (v, grad) in enumerate(((x, dx), (w, dw), (b, db))):
        step = torch.randn(v.shape, generator=g, device="cuda", dtype=torch.float64)
        args = [x.double(), w.double(), b.double()]
        at = lambda t: f(*[a + t * step if j == i else a for j, a in enumerate(args)])
        want = (at(1e-4) - at(-1e-4)) / 2e-4
        got = (grad.double() * step).sum()
        # third derivatives times 1e-8 and FP32 roundings of the gradient's terms
        assert abs(got - want) <= 1e-5 * (grad.double().abs() * step.abs()).sum() + 1e-6


def test_other_stream():
    x, w, b, dy = make(2000, 4096, BF, BF)
    want = lpq.layer_norm(x, w, b)
    back = lpq.layer_norm_backward(dy, x, want[1], want[2], w)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = lpq.layer_norm(x, w, b, stream=s)
    gback = lpq.layer_norm_backward(dy, x, got[1], got[2], w, stream=s)
    junk = [torch.full((2000, 4096), 1.0, device="cuda") for _ in range(4)]  # would take over freed scratch
    s.synchronize()
    for p, q in zip(want + back, got + gback):
        assert torch.equal(p, q)
    del junk


@pytest.mark.parametrize("dt", [BF])
def test_offsets_beyond_32_bits(dt):
    """Over 2^31 elements: the last rows are as right as the first."""
    rows, cols = (1 << 31) // 8192 + 40, 8192
    w, b = torch.ones(cols, dtype=dt, device="cuda"), torch.zeros(cols, dtype=dt, device="cuda")
    x = torch.empty(rows, cols, dtype=dt, device="cuda").normal_()
    y, mean, rstd = lpq.layer_norm(x, w, b)
    for part in (slice(0, 8), slice(rows - 8, rows)):
        check_forward(x[part], w, b, 1e-5, y[part], mean[part], rstd[part])
    dx, _, db = lpq.layer_norm_backward(y, x, mean, rstd, w)
    for part in (slice(0, 8), slice(rows - 8, rows)):
        check_backward(y[part], x[part], w, mean[part], rstd[part], dx[part], None, None)


def test_python_refusals():
    x, w, b, dy = make(4, 64, BF, BF)
    with pytest.raises(AssertionError):
        lpq.layer_norm(x.half(), w, b)
    with pytest.raises(AssertionError):
        lpq.layer_norm(x.T, None, None)
    with pytest.raises(AssertionError):
        lpq.layer_norm(x, w.float(), b)
    with pytest.raises(AssertionError):
        lpq.layer_norm(x, w[:32], b)
    with pytest.raises(lpq.LpqError) as e:
        lpq.layer_norm(x[:1].expand(4, 64), w, b)
    assert e.value.status == lpq.ERR_SHAPE
    with pytest.raises(lpq.LpqError) as e:
        lpq.layer_norm(x, w, b, eps=-1.0)
    assert e.value.status == lpq.ERR_INVALID_ARG
