"""The matrix-vector product's ways of working: x as f16 or (where its range is
too wide for that) bf16 operands, segments of K joined in a CTA or a cluster,
MXFP4 groups beyond f16's range, the longest sums."""
import pytest
import torch

from precision_transformer_gemms_gb300 import lpq, synth
from test_gpu_matvec import FORMATS, check, quantized

pytestmark = pytest.mark.gpu


def wide_x(m, k, seed):
    """Values over 2^-100 .. 2^60 in some runs of 512, ordinary ones elsewhere."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = torch.randn(m, k, generator=g, device="cuda")
    e = torch.randint(-100, 60, (m, k), generator=g, device="cuda").float()
    run = torch.arange(k, device="cuda") // 512 % 3 == 1
    return torch.where(run, x * torch.exp2(e), x).bfloat16()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("layout", [lpq.SF_GEMM, lpq.SF_PLAIN])
@pytest.mark.parametrize("n,k", [(256, 512), (384, 2048), (144, 4096), (25600, 4096), (640, 16384), (96, 1056)])
@pytest.mark.parametrize("m", [1, 2, 5, 8])
def test_segments_and_wide_x(n, k, m, fmt, layout):
    w = quantized(n, k, fmt, layout, seed=k + n)
    x = synth.bf16_normal((m, k), 1.0, m, "cuda")
    check(x, w, lpq.matvec(x, w, out_fp32=True))
    x = wide_x(m, k, m)
    check(x, w, lpq.matvec(x, w, out_fp32=True))


@pytest.mark.parametrize("n,k", [(512, 4096), (25600, 4096)])
@pytest.mark.parametrize("fmt", [lpq.NVFP4, lpq.MXFP4])
def test_a_row_and_a_token_stand_alone(n, k, fmt):
    """A result depends not on the other rows, nor on other tokens of ordinary range
    (a token whose range takes bf16 operands has the others' products added in
    another order)."""
    w = quantized(25600, k, fmt)
    part = lpq.Copy.of_parts(fmt, n, k, w.codes, w.scales, w.tensor_scale)
    plain = synth.bf16_normal((5, k), 1.0, 3, "cuda")
    for x in (plain, torch.cat((plain, wide_x(1, k, 4)))):
        y = lpq.matvec(x, w, out_fp32=True)
        assert torch.equal(lpq.matvec(x, part, out_fp32=True), y[:, :n])
    y = lpq.matvec(plain, part, out_fp32=True)
    for i in range(5):
        assert torch.equal(lpq.matvec(plain[i:i + 1], part, out_fp32=True), y[i:i + 1])


@pytest.mark.parametrize("n,k", [(256, 1024), (200, 4096), (20480, 4096)])
@pytest.mark.parametrize("wide", [False, True])
def test_mxfp4_groups_of_any_size(n, k, wide):
    """Scales over all of E8M0's range that keeps the products finite, mixed in one matrix."""
    g = torch.Generator(device="cuda")
    g.manual_seed(n)
    groups = k // 32
    codes = torch.randint(0, 256, (n, k // 2), generator=g, device="cuda", dtype=torch.uint8)
    scales = torch.randint(110, 130, (n, groups), generator=g, device="cuda")
    far = torch.rand(n, groups, generator=g, device="cuda") < 0.05
    # (up to 2^92 against x of ordinary size, up to 2^60 against x up to 2^62)
    scales = torch.where(far, torch.randint(0, 187 if wide else 220, (n, groups), generator=g, device="cuda"), scales).to(torch.uint8)
    zero = torch.rand(n, groups, generator=g, device="cuda") < 0.05
    codes.view(n, groups, 16)[zero] = 0
    scales[zero] = 0
    w = lpq.Copy.of_parts(lpq.MXFP4, n, k, codes.view(-1), scales.view(-1), None, lpq.SF_PLAIN)
    full = torch.zeros(-(-n // 128) * 128, -(-groups // 8) * 8, dtype=torch.uint8, device="cuda")
    full[:n, :groups] = scales
    tiled = full.view(-1, 4, 32, full.shape[1] // 4, 4).permute(0, 3, 2, 1, 4).contiguous().view(-1)
    same = lpq.Copy.of_parts(lpq.MXFP4, n, k, codes.view(-1), tiled, None, lpq.SF_GEMM)
    x = wide_x(2, k, 2) if wide else synth.bf16_normal((3, k), 1.0, 1, "cuda")
    check(x, same, lpq.matvec(x, same, out_fp32=True))
    check(x, w, lpq.matvec(x, w, out_fp32=True))


@pytest.mark.parametrize("k,layout", [(65536, lpq.SF_PLAIN), (65536, lpq.SF_GEMM), (1 << 19, lpq.SF_GEMM), ((1 << 19) - 32, lpq.SF_GEMM)])
@pytest.mark.parametrize("fmt", [lpq.NVFP4, lpq.MXFP4])
def test_longest_sums(k, layout, fmt):
    w = quantized(48, k, fmt, layout)
    x = synth.bf16_normal((3, k), 1.0, 5, "cuda")
    check(x, w, lpq.matvec(x, w, out_fp32=True))


def test_many_passes():
    w = quantized(160, 224, lpq.NVFP4)
    x = synth.bf16_normal((1003, 224), 1.0, 5, "cuda")
    check(x, w, lpq.matvec(x, w))
