"""Groups of zero codes add 0 whatever (finite) scale stands beside them."""
import pytest
import torch

from precision_transformer_gemms_gb300 import lpq, synth
from test_gpu_matvec import check
from test_gpu_matvec_paths import wide_x

pytestmark = pytest.mark.gpu


def copies(fmt, codes, scales, ts):
    """The weights with plain scales and with the tensor cores' layout of them."""
    n, groups = scales.shape
    k = codes.shape[1] * 2
    per = 8 if fmt == lpq.MXFP4 else 16  # blocks of 256 columns
    full = torch.zeros(-(-n // 128) * 128, -(-groups // per) * per, dtype=torch.uint8, device="cuda")
    full[:n, :groups] = scales
    tiled = full.view(-1, 4, 32, full.shape[1] // 4, 4).permute(0, 3, 2, 1, 4).contiguous().view(-1)
    return [lpq.Copy.of_parts(fmt, n, k, codes.view(-1), scales.reshape(-1), ts, lpq.SF_PLAIN),
            lpq.Copy.of_parts(fmt, n, k, codes.view(-1), tiled, ts, lpq.SF_GEMM)]


@pytest.mark.parametrize("fmt,scales", [(lpq.MXFP4, 255), (lpq.NVFP4, 127)])
@pytest.mark.parametrize("k", [64, 512, 4096])
@pytest.mark.parametrize("m", [1, 3, 8])
@pytest.mark.parametrize("wide", [False, True])
def test_zero_rows_for_every_scale(fmt, scales, k, m, wide):
    """A row of zero codes (of either sign) for every scale byte that is a number."""
    blk = 32 if fmt == lpq.MXFP4 else 16
    codes = torch.randint(0, 2, (scales, k // 2), dtype=torch.uint8, device="cuda") * 0x88
    sf = torch.arange(scales, device="cuda").to(torch.uint8)[:, None].expand(scales, k // blk).contiguous()
    ts = torch.ones(1, device="cuda") if fmt != lpq.MXFP4 else None
    x = wide_x(m, k, m) if wide else synth.bf16_normal((m, k), 1.0, m, "cuda")
    for w in copies(fmt, codes, sf, ts):
        assert not lpq.matvec(x, w, out_fp32=True).any()


@pytest.mark.parametrize("n,k", [(256, 1024), (200, 4096), (20480, 4096)])
@pytest.mark.parametrize("wide", [False, True])
def test_zero_groups_among_others(n, k, wide):
    g = torch.Generator(device="cuda")
    g.manual_seed(n + k)
    codes = torch.randint(0, 256, (n, k // 2), generator=g, device="cuda", dtype=torch.uint8)
    sf = torch.randint(110, 130, (n, k // 32), generator=g, device="cuda")
    zero = torch.rand(n, k // 32, generator=g, device="cuda") < 0.1
    codes.view(n, k // 32, 16)[zero] = 0
    sf = torch.where(zero, torch.randint(0, 255, (n, k // 32), generator=g, device="cuda"), sf).to(torch.uint8)
    x = wide_x(2, k, 5) if wide else synth.bf16_normal((2, k), 1.0, 5, "cuda")
    for w in copies(lpq.MXFP4, codes, sf, None):
        check(x, w, lpq.matvec(x, w, out_fp32=True))
