"""Copy.of_parts refuses what a kernel would read past: the checks are made on the
host and nothing is launched."""
import types

import pytest
import torch

from precision_transformer_gemms_gb300 import lpq

FORMATS = [lpq.NVFP4, lpq.NVFP4_2D, lpq.MXFP4, lpq.MXFP8, lpq.FP8_E4M3, lpq.FP8_BLOCK_1x128, lpq.FP8_BLOCK_128x128, lpq.BF16]


def parts(fmt, rows, cols, layout, device="cpu"):
    """Buffers of exactly the sizes that the copy has."""
    c = lpq.Copy(fmt, rows, cols, False, layout, device)
    return dict(codes=c.codes, scales=c.scales, tensor_scale=c.tensor_scale)


def of(fmt, rows, cols, layout, p):
    return lpq.Copy.of_parts(fmt, rows, cols, p["codes"], p["scales"], p["tensor_scale"], layout)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("layout", [lpq.SF_PLAIN, lpq.SF_GEMM])
def test_refusals(fmt, layout):
    if fmt == lpq.BF16 and layout == lpq.SF_GEMM:
        pytest.skip("no scales")
    rows, cols = 256, 512
    good = parts(fmt, rows, cols, layout)
    # host tensors of the right sizes: everything but the device is as it should be
    with pytest.raises(AssertionError, match="one CUDA device"):
        of(fmt, rows, cols, layout, good)
    for name in good:
        t = good[name]
        if t is None:
            continue
        flat = t.view(-1)
        for bad in (None, flat[:-1], flat.to(torch.float64), torch.stack((flat, flat), 1)[:, 0]):
            if name == "tensor_scale" and bad is not None and bad.numel() == 1 and bad.is_contiguous() and bad.dtype is torch.float32:
                continue  # (one element is contiguous whatever its stride)
            with pytest.raises(AssertionError, match=name):
                of(fmt, rows, cols, layout, {**good, name: bad})


def test_scales_of_the_other_layout():
    """Plain scales are fewer bytes than the tensor-core layout's, which is padded."""
    for fmt in (lpq.NVFP4, lpq.MXFP4):
        p = parts(fmt, 200, 352, lpq.SF_PLAIN)
        with pytest.raises(AssertionError, match="scales"):
            of(fmt, 200, 352, lpq.SF_GEMM, p)


def test_unknown_format_and_layout():
    p = parts(lpq.NVFP4, 32, 64, lpq.SF_GEMM)
    for fmt, layout in ((99, lpq.SF_GEMM), (lpq.NVFP4, 7)):
        with pytest.raises(lpq.LpqError):
            of(fmt, 32, 64, layout, p)


def test_products_of_tokens_elsewhere_are_refused():
    x = types.SimpleNamespace(shape=(1, 64), dtype=torch.bfloat16, get_device=lambda: 0)
    with pytest.raises(AssertionError, match="where the weights"):
        lpq.matvec(x, lpq.Copy(lpq.NVFP4, 32, 64, False, device="cpu"))


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("layout", [lpq.SF_PLAIN, lpq.SF_GEMM])
def test_accepts_a_copys_own_parts(fmt, layout):
    if fmt == lpq.BF16 and layout == lpq.SF_GEMM:
        pytest.skip("no scales")
    p = parts(fmt, 256, 512, layout, "cuda")
    c = of(fmt, 256, 512, layout, p)
    assert c.view().codes == p["codes"].data_ptr()
    for name in p:  # one of them on the host
        if p[name] is not None:
            with pytest.raises(AssertionError, match="one CUDA device"):
                of(fmt, 256, 512, layout, {**p, name: p[name].cpu()})
