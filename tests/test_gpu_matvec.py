"""Products of a few tokens with 4-bit weights against the definition in 64 bits.

Tolerance: codes times scales are exact in the kernels' operands, so only the
FP32 sum rounds.  In any order it is off by at most (additions in a row) x
2^-23 of sum |x w|; K / 16 + 64 consecutive additions cover every kernel (the
tensor core adds 16 products at once).  bf16 outputs add 2^-8 of the value."""
import numpy as np
import pytest
import torch

from lpq_testutil import plain_scales
from precision_transformer_gemms_gb300 import lpq, synth

pytestmark = pytest.mark.gpu
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
FORMATS = [lpq.NVFP4, lpq.NVFP4_2D, lpq.MXFP4]


def e4m3(c):
    c = c.astype(np.int64) & 127
    v = np.where(c < 8, (c & 7) * 2.0 ** -9, (8 + (c & 7)) * 2.0 ** ((c >> 3) - 10.0))
    return np.where(c == 127, np.nan, v)


def dequantized(w):
    """The weights a copy stands for, without its tensor scale, in 64 bits."""
    codes = w.codes_matrix().cpu().numpy()
    q = np.stack((codes & 15, codes >> 4), -1).reshape(w.rows, w.cols)
    val = np.array(E2M1 + [-v for v in E2M1])[q]
    s = plain_scales(w)
    if w.fmt == lpq.MXFP4:
        s = np.where(s == 255, np.nan, 2.0 ** (s.astype(np.float64) - 127))
    else:
        s = e4m3(s)
    blk = w.cols // s.shape[1]
    return val * np.repeat(s, blk, 1)


def check(x, w, y):
    d = torch.from_numpy(dequantized(w)).cuda()
    ts = w.tensor_scale.double().item() if w.fmt != lpq.MXFP4 else 1.0
    want = x.double() @ d.T * ts
    k = w.cols / 16 + 64
    tol = k * 2.0 ** -23 * (x.double().abs() @ d.abs().T) * ts + (2.0 ** -8 if y.dtype == torch.bfloat16 else 2.0 ** -22) * want.abs()
    err = (y.double() - want).abs()
    assert torch.all(err <= tol + 1e-38), float((err / (tol + 1e-38)).max())


def quantized(n, k, fmt, layout=lpq.SF_GEMM, seed=0, std=0.02):
    w = synth.bf16_normal((n, k), std, seed, "cuda", 0.01, 20.0)
    return lpq.quantize(w, fmt, lpq.ROWWISE, sf_layout=layout).row


SHAPES = [(16, 32), (48, 64), (16, 96), (80, 160), (128, 256), (384, 512), (1008, 288), (144, 4096), (4096, 128), (2000, 1056), (64, 16384),
          (272, 8224)]


@pytest.mark.parametrize("n,k", SHAPES)
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("layout", [lpq.SF_GEMM, lpq.SF_PLAIN])
def test_sizes(n, k, fmt, layout):
    w = quantized(n, k, fmt, layout, seed=n + k)
    for m in (1, 3):
        x = synth.bf16_normal((m, k), 1.0, m, "cuda", 0.01, 30.0)
        check(x, w, lpq.matvec(x, w))
    check(x, w, lpq.matvec(x, w, out_fp32=True))


@pytest.mark.parametrize("m", [1, 2, 3, 4, 5, 6, 7, 8, 9, 15, 16, 17, 31, 40])
@pytest.mark.parametrize("fmt", [lpq.NVFP4, lpq.MXFP4])
def test_tokens(m, fmt):
    w = quantized(336, 1440, fmt)
    x = synth.bf16_normal((m, 1440), 1.0, m, "cuda")
    y = lpq.matvec(x, w, out_fp32=True)
    check(x, w, y)
    assert y.shape == (m, 336) and y.dtype == torch.float32


@pytest.mark.parametrize("n", [1, 2, 15, 17, 31, 33, 100, 127, 129, 255, 1001])
def test_any_number_of_rows(n):
    """Copies of weights whose row count is no multiple of anything."""
    for fmt in (lpq.NVFP4, lpq.MXFP4):
        w = quantized(n, 224, fmt)
        x = synth.bf16_normal((2, 224), 1.0, 7, "cuda")
        check(x, w, lpq.matvec(x, w))


def test_every_code_and_scale():
    """All 16 codes against all scales that stand for numbers, exactly: x picks one weight at a time."""
    k = 256
    for fmt, scales in ((lpq.NVFP4, range(127)), (lpq.MXFP4, range(0, 252))):
        n = len(scales)
        codes = torch.randint(0, 256, (n, k // 2), dtype=torch.uint8, device="cuda")
        codes[:, :8] = torch.arange(16, device="cuda").view(8, 2).mul(torch.tensor([1, 16], device="cuda")).sum(1).to(torch.uint8)
        blk = 32 if fmt == lpq.MXFP4 else 16
        sf = torch.tensor(list(scales), dtype=torch.uint8, device="cuda")[:, None].expand(n, k // blk).contiguous()
        one = torch.ones(1, device="cuda") if fmt != lpq.MXFP4 else None
        w = lpq.Copy.of_parts(fmt, n, k, codes.view(-1), sf.view(-1), one, lpq.SF_PLAIN)
        x = torch.zeros(16, k, dtype=torch.bfloat16, device="cuda")
        x[torch.arange(16), torch.arange(16)] = 1.0
        y = lpq.matvec(x, w, out_fp32=True)
        want = torch.from_numpy(dequantized(w)).cuda()[:, :16].T
        assert torch.equal(y.double(), want)


def test_special_values():
    w = quantized(64, 128, lpq.NVFP4)
    x = synth.bf16_normal((3, 128), 1.0, 1, "cuda")
    x[1, 3] = float("nan")
    x[2] = 0.0
    y = lpq.matvec(x, w, out_fp32=True)
    check(x[:1], w, y[:1])
    assert y[1].isnan().all() and not y[2].any()
    # values far apart: the small ones count where the large one meets a zero weight
    codes = torch.full((1, 64), 0x22, dtype=torch.uint8, device="cuda")
    codes[0, 0] = 0x20
    sf = torch.full((1, 8), 0x38, dtype=torch.uint8, device="cuda")
    one = lpq.Copy.of_parts(lpq.NVFP4, 1, 128, codes.view(-1), sf.view(-1), torch.ones(1, device="cuda"), lpq.SF_PLAIN)
    x = torch.ones(1, 128, dtype=torch.bfloat16, device="cuda")
    x[0, 0] = 1e30
    assert lpq.matvec(x, one, out_fp32=True).item() == 127.0
    # a scale that is no number reaches its row only
    sf = torch.full((2, 8), 0x38, dtype=torch.uint8, device="cuda")
    sf[1, 2] = 0x7F
    two = lpq.Copy.of_parts(lpq.NVFP4, 2, 128, codes.expand(2, 64).contiguous().view(-1), sf.view(-1), torch.ones(1, device="cuda"), lpq.SF_PLAIN)
    y = lpq.matvec(torch.ones(1, 128, dtype=torch.bfloat16, device="cuda"), two)
    assert y[0, 0].item() == 127.0 and y[0, 1].isnan()
    sf = torch.full((2, 4), 127, dtype=torch.uint8, device="cuda")
    sf[0, 3] = 255
    mx = lpq.Copy.of_parts(lpq.MXFP4, 2, 128, codes.expand(2, 64).contiguous().view(-1), sf.view(-1), None, lpq.SF_PLAIN)
    y = lpq.matvec(torch.ones(1, 128, dtype=torch.bfloat16, device="cuda"), mx)
    assert y[0, 0].isnan() and y[0, 1].item() == 127.0


def test_empty():
    w = quantized(32, 64, lpq.NVFP4)
    assert lpq.matvec(torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"), w).shape == (0, 32)
    none = lpq.Copy.of_parts(lpq.NVFP4, 32, 0, w.codes, w.scales, w.tensor_scale)
    y = lpq.matvec(torch.empty(2, 0, dtype=torch.bfloat16, device="cuda"), none)
    assert y.shape == (2, 32) and not y.any()
    none = lpq.Copy.of_parts(lpq.NVFP4, 0, 64, w.codes, w.scales, w.tensor_scale)
    assert lpq.matvec(torch.empty(2, 64, dtype=torch.bfloat16, device="cuda"), none).shape == (2, 0)


def test_strided_tokens_and_other_stream():
    w = quantized(512, 1024, lpq.MXFP4)
    big = synth.bf16_normal((6, 2048), 1.0, 1, "cuda")
    x = big[::2, 512:1536]
    want = lpq.matvec(x.contiguous(), w)
    assert torch.equal(lpq.matvec(x, w), want)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = lpq.matvec(x, w, stream=s)
    s.synchronize()
    assert torch.equal(got, want)


def test_reproducible():
    w = quantized(4096, 4096, lpq.NVFP4)
    x = synth.bf16_normal((5, 4096), 1.0, 1, "cuda")
    y = lpq.matvec(x, w, out_fp32=True)
    for _ in range(3):
        assert torch.equal(lpq.matvec(x, w, out_fp32=True), y)


def test_offsets_beyond_32_bits():
    """Over 2^32 bytes of codes: the last rows are as right as the first."""
    k, part = 16384, 4096
    n = (1 << 33) // k + 128  # 4 GiB of codes and one group more
    w = quantized(part, k, lpq.NVFP4)
    per = w.scales.numel() // (part // 128)
    codes = w.codes.view(part, -1).repeat(-(-n // part), 1)[:n].contiguous()
    scales = w.scales.view(part // 128, per).repeat(-(-n // part), 1)[: n // 128].contiguous()
    big = lpq.Copy.of_parts(lpq.NVFP4, n, k, codes.view(-1), scales.view(-1), w.tensor_scale)
    x = synth.bf16_normal((2, k), 1.0, 3, "cuda")
    y, want = lpq.matvec(x, big), lpq.matvec(x, w)
    check(x, w, want)
    reps = torch.arange(n, device="cuda") % part
    assert torch.equal(y, want[:, reps])


def test_python_refusals():
    w = quantized(32, 64, lpq.NVFP4)
    x = torch.ones(1, 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(AssertionError):
        lpq.matvec(x.float(), w)
    with pytest.raises(AssertionError):
        lpq.matvec(x[:, :32], w)
    with pytest.raises(lpq.LpqError) as e:
        lpq.matvec(x, lpq.quantize(torch.ones(32, 64, dtype=torch.bfloat16, device="cuda"), lpq.MXFP8, lpq.ROWWISE).row)
    assert e.value.status == lpq.ERR_UNSUPPORTED
