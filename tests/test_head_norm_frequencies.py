"""The library's array of frequencies: kept by value, whatever kind of number the base is."""
import numpy
import pytest
import torch

from precision_transformer_gemms_gb300 import lpq


def test_a_base_that_is_changed_in_place_is_another_base():
    base = torch.tensor(10000.0, dtype=torch.float64)
    first = list(lpq._frequencies(64, base, None))
    base.fill_(500000.0)
    second = list(lpq._frequencies(64, base, None))
    assert first == [10000.0 ** (-2.0 * i / 64) for i in range(32)]
    assert second == [500000.0 ** (-2.0 * i / 64) for i in range(32)]


def test_frequencies_of_any_kind():
    own = torch.tensor([1.0, 0.5, 0.25])
    assert list(lpq._frequencies(6, 10000.0, own)) == [1.0, 0.5, 0.25]
    own[1] = 0.75
    assert list(lpq._frequencies(6, 10000.0, own)) == [1.0, 0.75, 0.25]
    assert list(lpq._frequencies(6, 10000.0, numpy.array([3.0, 2.0, 1.0]))) == [3.0, 2.0, 1.0]
    assert lpq._frequencies(64, numpy.float64(10000.0), None) is lpq._frequencies(64, 10000, None)


@pytest.mark.gpu
def test_the_angles_follow_the_base():
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    x, dy = (torch.randn(4, 192, generator=g, device="cuda") for _ in range(2))
    positions = torch.tensor([0, 5, 1000, 77], device="cuda")
    base = torch.tensor(10000.0)
    for value in (10000.0, 500000.0, 200.0):
        base.fill_(value)
        assert torch.equal(lpq.qk_norm_rope(x, 2, 1, 64, positions, base=base), lpq.qk_norm_rope(x, 2, 1, 64, positions, base=value))
        got, want = (lpq.qk_norm_rope_backward(dy, x, 2, 1, 64, positions, base=b)[0] for b in (base, value))
        assert torch.equal(got, want)
