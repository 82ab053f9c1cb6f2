"""The language head: its operators together, as a training step and as decoding."""
import importlib.util
import os

import pytest
import torch

from precision_transformer_gemms_gb300 import lpq
from precision_transformer_gemms_gb300.head import LanguageHead

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def make(t=300, d=256, v=1111, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")
    head = LanguageHead((1 + 0.1 * r(d)).bfloat16(), (0.1 * r(d)).bfloat16(), (0.05 * r(v, d)).bfloat16())
    labels = torch.randint(0, v, (t,), generator=g, device="cuda")
    labels[::9] = -100
    return head, r(t, d).bfloat16(), labels


@pytest.mark.parametrize("stream", [False, True])
def test_training_step_against_autograd(stream):
    """Loss and all four gradients against differentiation in 64 bits.  The norm's
    bf16 output carries 2^-8 of each hidden value into everything behind it, dl and
    dh 2^-8 each: 3 * 2^-8 of a gradient's norm, doubled for their spread."""
    head, x, labels = make()
    s = torch.cuda.Stream() if stream else None
    torch.cuda.synchronize()
    loss, saved = head.loss(x, labels, stream=s)
    grads = head.backward(saved, stream=s)
    torch.cuda.synchronize()
    p = [t.double().requires_grad_() for t in (x, head.weight, head.bias, head.w)]
    h = torch.nn.functional.layer_norm(p[0], (256,), p[1], p[2], head.eps)
    want = torch.nn.functional.cross_entropy(h @ p[3].T, labels)
    assert abs(loss.item() - want.item()) <= 2.0 ** -8 * want.item()
    for name, g in zip(("x", "weight", "bias", "w"), torch.autograd.grad(want, p)):
        assert (grads[name].double() - g).norm() <= 6 * 2.0 ** -8 * g.norm(), name


def test_no_row_with_a_target():
    head, x, labels = make(t=40)
    loss, saved = head.loss(x, torch.full_like(labels, -100))
    assert loss.item() == 0
    for g in head.backward(saved).values():
        assert not g.any()


@pytest.mark.parametrize("fmt", [lpq.NVFP4, lpq.MXFP4])
def test_decoding_uses_the_quantized_weights(fmt):
    head, x, _ = make(t=5, v=1104)
    with pytest.raises(AssertionError):
        head.logits(x)
    y = head.freeze(fmt).logits(x)
    h, _, _ = lpq.layer_norm(x, head.weight, head.bias)
    assert torch.equal(y, lpq.matvec(h, head.frozen, out_fp32=True))
    # 4-bit weights: at most a sixth of a block's largest value away (half the grid's widest
    # step, 2 of 6), about a fifteenth of the typical one: the logits keep their direction
    full = h.float() @ head.w.float().T
    assert torch.nn.functional.cosine_similarity(y, full, dim=1).min() > 0.97


def test_prompt_logits_scale_with_the_norms_amax():
    head, x, _ = make(t=256, v=1104)
    head.freeze()
    h, _, _ = lpq.layer_norm(x, head.weight, head.bias)
    want = lpq.gemm(lpq.FPROP, lpq.quantize(h, lpq.NVFP4, lpq.ROWWISE).row, head.frozen, out_fp32=True)
    assert torch.equal(head.prompt_logits(x), want)


@pytest.mark.parametrize("fmt", [lpq.NVFP4, lpq.MXFP4])
def test_example(fmt):
    spec = importlib.util.spec_from_file_location("language_head", os.path.join(ROOT, "examples", "language_head.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    first, last, right, prompt = m.train_and_decode(steps=40, fmt=fmt, say=lambda *_: None)
    assert first > 6.5 and last < 0.5 * first and right > 0.9  # ln 1000 = 6.9 untrained
    assert prompt is None or prompt > 0.9
