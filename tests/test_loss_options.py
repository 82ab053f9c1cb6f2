"""Options of the loss's backward pass: refusals and workspace sizes, decided on the host."""
import ctypes

import pytest

from precision_transformer_gemms_gb300 import lpq

A = 1 << 20  # an aligned address that is never read


def back(opts, t=4, wsb=1 << 30):
    return lpq.lib().lpq_linear_ce_backward_ex(A, 64, A, 64, A, A, A, t, 100, 64, A, A, 0, 0, A, wsb, opts, None)


@pytest.mark.parametrize("opts", [lpq.CeOpts(two_terms=2), lpq.CeOpts(two_terms=-1), lpq.CeOpts(reserved=(ctypes.c_int32 * 3)(0, 1, 0))])
def test_refusals(opts):
    assert back(ctypes.byref(opts)) == lpq.ERR_INVALID_ARG and lpq.last_error()


def size(t, v, d, backward, piece=0):
    n = ctypes.c_size_t()
    assert lpq.lib().lpq_linear_ce_workspace(t, v, d, backward, piece, ctypes.byref(n)) == lpq.OK
    return n.value


def test_workspace():
    # room for the second terms of all rows; few rows have it either way
    assert size(4096, 5000, 64, 2, 1024) >= size(4096, 5000, 64, 1, 1024) + (4096 - 128) * 1024 * 2
    assert size(128, 5000, 64, 2) == size(128, 5000, 64, 1)
    assert size(65536, 131072, 4096, 2) <= 1.2 * size(65536, 131072, 4096, 1)  # the pieces are half as wide
    one = size(4096, 100, 64, 1)
    assert size(4096, 100, 64, 2) > one
    opts = lpq.CeOpts(two_terms=1)
    assert back(ctypes.byref(opts), t=4096, wsb=one) == lpq.ERR_INVALID_ARG
