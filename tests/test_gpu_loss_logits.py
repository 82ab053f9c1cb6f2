"""The backward pass's logits are the forward's, to the last bit: where a row has
no other word to be, exp(l - lse) is 1 and its gradients are 0 exactly."""
import pytest
import torch

from precision_transformer_gemms_gb300 import lpq

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("t", [1, 40, 128, 129, 300])
@pytest.mark.parametrize("d", [64, 1024, 1032, 2056, 4096, 8200])
@pytest.mark.parametrize("v", [1, 300])
def test_certain_words_have_no_gradient(t, d, v):
    g = torch.Generator(device="cuda")
    g.manual_seed(t + d)
    # positive values: the sums grow from step to step, as those that the tensor core cuts most
    h = torch.rand(t, d, generator=g, device="cuda").bfloat16()
    w = (200.0 / d * torch.rand(v, d, generator=g, device="cuda") - 1000.0 / d).bfloat16()
    word = v // 2
    w[word] = (100.0 / d * torch.rand(d, generator=g, device="cuda")).bfloat16()  # others lie over 150 below
    labels = torch.full((t,), word, device="cuda")
    if t > 1:
        labels[t // 2] = -100  # (a row without target moves the others)
    loss, lse = lpq.linear_cross_entropy(h, w, labels)
    assert not loss.any()
    dh, dw = lpq.linear_cross_entropy_backward(h, w, labels, lse, torch.ones(t, device="cuda"), out_fp32=True)
    assert not dh.any() and not dw.any()
