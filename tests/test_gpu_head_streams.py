"""The head on a stream other than the current one, which has work of its own
pending: every step, frozen weights included, is ordered on the stream given."""
import pytest
import torch

from precision_transformer_gemms_gb300 import lpq
from precision_transformer_gemms_gb300.head import LanguageHead
from test_gpu_head import make
from test_gpu_streams import pool_of

pytestmark = pytest.mark.gpu


def busy(sizes=()):
    """Pending work on the current stream, and blocks given back that it still writes."""
    torch.cuda._sleep(30_000_000)
    for n in sizes:
        torch.full((n,), 7, dtype=torch.uint8, device="cuda").add_(1)


@pytest.mark.parametrize("strided", [False, True])
def test_freeze_and_decode(strided):
    head, x, _ = make(t=256, v=1104)
    if strided:  # (the quantizer takes a copy)
        w = torch.empty(1104, 512, dtype=torch.bfloat16, device="cuda")[:, ::2]
        w.copy_(head.w)
        head = LanguageHead(head.weight, head.bias, w)
    head.freeze()
    frozen = [t.clone() for t in lpq._tensors(head.frozen)]
    logits, prompt = head.logits(x[:3]), head.prompt_logits(x)
    sizes = [t.nbytes for t in lpq._tensors(head.frozen)] + [logits.nbytes, prompt.nbytes, x.nbytes, head.w.numel() * 2]
    head.frozen = None
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    busy(sizes)
    head.freeze(stream=s)
    got = list(lpq._tensors(head.frozen))
    got_logits, got_prompt = head.logits(x[:3], stream=s), head.prompt_logits(x, stream=s)
    s.synchronize()
    assert torch.equal(got_logits, logits) and torch.equal(got_prompt, prompt)
    torch.cuda.synchronize()
    for a, b in zip(got, frozen):
        assert torch.equal(a, b)
        assert pool_of(a) == s.cuda_stream
    assert pool_of(got_logits) == pool_of(got_prompt) == s.cuda_stream


def test_training_step():
    head, x, labels = make()
    loss, saved = head.loss(x, labels)
    grads = head.backward(saved)
    sizes = [t.nbytes for t in lpq._tensors((loss, saved, grads))]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    busy(sizes)
    got_loss, got_saved = head.loss(x, labels, stream=s)
    got = head.backward(got_saved, stream=s)
    s.synchronize()
    assert torch.equal(got_loss, loss) and pool_of(got_loss) == s.cuda_stream
    for name in grads:
        assert torch.equal(got[name], grads[name]) and pool_of(got[name]) == s.cuda_stream
