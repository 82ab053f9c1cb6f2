"""What an Adapters object holds cannot change unseen between its making and a call."""
import pytest
import torch

from precision_transformer_gemms_gb300 import lpq
from test_gpu_adapters import check, make

pytestmark = pytest.mark.gpu


def test_its_tensors_cannot_be_replaced():
    _, ad, _, _ = make(64, 64, 8, 2, 2, lpq.NVFP4)
    for name in ("a", "b", "scale", "count", "rank", "k", "rows", "device"):
        with pytest.raises(AttributeError):
            setattr(ad, name, getattr(ad, name))


def test_memory_that_moves_is_followed():
    w, ad, index, x = make(96, 128, 16, 3, 5, lpq.MXFP4)
    _, other, _, _ = make(96, 128, 16, 3, 5, lpq.MXFP4, seed=9)
    kept = ad.a.clone(), ad.b.clone(), ad.scale.clone()
    for mine, new in ((ad.a, other.a), (ad.b, other.b), (ad.scale, other.scale)):
        mine.data = new
        check(x, w, ad, index, lpq.matvec(x, w, adapters=ad, index=index))
    assert not any(torch.equal(k, t) for k, t in zip(kept, (ad.a, ad.b, ad.scale)))
