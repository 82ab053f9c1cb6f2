"""A prompt through a head frozen in any 4-bit format that the GEMM takes."""
import pytest
import torch

from precision_transformer_gemms_gb300 import lpq
from test_gpu_head import make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt,acts", [(lpq.NVFP4, lpq.NVFP4), (lpq.NVFP4_2D, lpq.NVFP4), (lpq.MXFP4, lpq.MXFP4)])
def test_prompt_logits(fmt, acts):
    head, x, _ = make(t=256, v=1104)
    head.freeze(fmt)
    h, _, _ = lpq.layer_norm(x, head.weight, head.bias)
    want = lpq.gemm(lpq.FPROP, lpq.quantize(h, acts, lpq.ROWWISE).row, head.frozen, out_fp32=True)
    got = head.prompt_logits(x)
    assert torch.equal(got, want)
    full = h.float() @ head.w.float().T
    assert torch.nn.functional.cosine_similarity(got, full, dim=1).min() > 0.95  # 4-bit weights and activations


def test_prompt_needs_frozen_weights():
    head, x, _ = make(t=256, v=1104)
    with pytest.raises(AssertionError):
        head.prompt_logits(x)
