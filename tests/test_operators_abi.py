"""Argument checks of the norm, loss and matrix-vector entry points, and their
workspace sizes: all of it is decided on the host, without a GPU."""
import ctypes

import pytest

from precision_transformer_gemms_gb300 import lpq

A = 1 << 20  # an aligned address that is never read
VALID = (lpq.OK, lpq.ERR_ARCH, lpq.ERR_CUDA)  # arguments accepted: stops at the device check here


def norm(x=A, ldx=64, xt=0, w=A, b=A, wt=0, rows=4, cols=64, eps=1e-5, y=A, ldy=64, mean=A, rstd=A, amax=None):
    return lpq.lib().lpq_layer_norm(x, ldx, xt, w, b, wt, rows, cols, eps, y, ldy, mean, rstd, amax, None)


@pytest.mark.parametrize("kw,status", [
    (dict(xt=2), lpq.ERR_INVALID_ARG), (dict(wt=-1), lpq.ERR_INVALID_ARG), (dict(rows=-1), lpq.ERR_SHAPE),
    (dict(cols=0), lpq.ERR_SHAPE), (dict(ldx=63), lpq.ERR_SHAPE), (dict(ldy=0), lpq.ERR_SHAPE),
    (dict(eps=-1e-9), lpq.ERR_INVALID_ARG), (dict(eps=float("nan")), lpq.ERR_INVALID_ARG), (dict(x=None), lpq.ERR_INVALID_ARG),
    (dict(y=None), lpq.ERR_INVALID_ARG), (dict(x=A + 1), lpq.ERR_ALIGN), (dict(xt=1, y=A + 2), lpq.ERR_ALIGN),
    (dict(w=A + 1), lpq.ERR_ALIGN), (dict(wt=1, b=A + 2), lpq.ERR_ALIGN), (dict(mean=A + 2), lpq.ERR_ALIGN),
    (dict(amax=A + 1), lpq.ERR_ALIGN)])
def test_norm_refusals(kw, status):
    assert norm(**kw) == status
    assert lpq.last_error()


@pytest.mark.parametrize("kw", [dict(), dict(w=None, b=None), dict(mean=None, rstd=None), dict(x=A + 2, y=A + 6), dict(ldx=65, ldy=99),
                                dict(rows=0, x=None, y=None), dict(eps=0.0), dict(cols=1)])
def test_norm_accepts(kw):
    if lpq.torch.cuda.is_available():
        pytest.skip("the addresses are not memory")
    assert norm(**kw) in VALID


def norm_back(dy=A, lddy=64, x=A, ldx=64, xt=0, mean=A, rstd=A, w=A, wt=0, rows=4, cols=64, dx=A, lddx=64, dw=A, db=A, ws=A, wsb=1 << 30):
    return lpq.lib().lpq_layer_norm_backward(dy, lddy, x, ldx, xt, mean, rstd, w, wt, rows, cols, dx, lddx, dw, db, ws, wsb, None)


@pytest.mark.parametrize("kw,status", [
    (dict(xt=7), lpq.ERR_INVALID_ARG), (dict(lddy=3), lpq.ERR_SHAPE), (dict(lddx=63), lpq.ERR_SHAPE), (dict(mean=None), lpq.ERR_INVALID_ARG),
    (dict(rstd=None), lpq.ERR_INVALID_ARG), (dict(dx=None), lpq.ERR_INVALID_ARG), (dict(ws=None), lpq.ERR_INVALID_ARG),
    (dict(wsb=16), lpq.ERR_INVALID_ARG), (dict(ws=A + 4), lpq.ERR_ALIGN), (dict(dw=A + 1), lpq.ERR_ALIGN), (dict(dy=A + 1), lpq.ERR_ALIGN)])
def test_norm_backward_refusals(kw, status):
    assert norm_back(**kw) == status


def test_norm_workspace():
    n = ctypes.c_size_t(7)
    size = lambda r, c: (lpq.lib().lpq_layer_norm_workspace(r, c, ctypes.byref(n)), n.value)
    assert size(0, 64) == (0, 0)
    st, small = size(1, 64)
    assert st == 0 and small >= 2 * 64 * 4
    assert size(100000, 4096)[1] <= 64 << 20  # bounded, whatever the rows
    assert size(-1, 64)[0] == lpq.ERR_SHAPE
    assert lpq.lib().lpq_layer_norm_workspace(1, 1, None) == lpq.ERR_INVALID_ARG


def ce(h=A, ldh=64, w=A, ldw=64, labels=A, t=4, v=100, d=64, loss=A, lse=A, ws=A, wsb=1 << 30):
    return lpq.lib().lpq_linear_ce(h, ldh, w, ldw, labels, t, v, d, loss, lse, ws, wsb, None)


def ce_back(h=A, ldh=64, w=A, ldw=64, labels=A, lse=A, dloss=A, t=4, v=100, d=64, dh=A, dw=A, fp32=0, piece=0, ws=A, wsb=1 << 30):
    return lpq.lib().lpq_linear_ce_backward(h, ldh, w, ldw, labels, lse, dloss, t, v, d, dh, dw, fp32, piece, ws, wsb, None)


@pytest.mark.parametrize("kw,status", [
    (dict(t=-1), lpq.ERR_SHAPE), (dict(v=0), lpq.ERR_SHAPE), (dict(d=0), lpq.ERR_SHAPE), (dict(d=60), lpq.ERR_SHAPE),
    (dict(ldh=60), lpq.ERR_SHAPE), (dict(ldw=68), lpq.ERR_SHAPE), (dict(ldh=56), lpq.ERR_SHAPE), (dict(t=(1 << 30) + 1), lpq.ERR_SHAPE),
    (dict(h=None), lpq.ERR_INVALID_ARG), (dict(w=None), lpq.ERR_INVALID_ARG), (dict(labels=None), lpq.ERR_INVALID_ARG),
    (dict(h=A + 8), lpq.ERR_ALIGN), (dict(w=A + 2), lpq.ERR_ALIGN), (dict(labels=A + 4), lpq.ERR_ALIGN),
    (dict(ws=None), lpq.ERR_INVALID_ARG), (dict(wsb=0), lpq.ERR_INVALID_ARG), (dict(ws=A + 8), lpq.ERR_ALIGN), (dict(lse=A + 2), lpq.ERR_ALIGN)])
def test_loss_refusals(kw, status):
    assert ce(**kw) == status
    assert ce_back(**kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(loss=None), lpq.ERR_INVALID_ARG), (dict(lse=None), lpq.ERR_INVALID_ARG), (dict(loss=A + 2), lpq.ERR_ALIGN)])
def test_loss_forward_refusals(kw, status):
    assert ce(**kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(dloss=None), lpq.ERR_INVALID_ARG), (dict(dh=None), lpq.ERR_INVALID_ARG), (dict(dw=None), lpq.ERR_INVALID_ARG),
    (dict(fp32=2), lpq.ERR_INVALID_ARG), (dict(piece=-64), lpq.ERR_SHAPE), (dict(piece=96), lpq.ERR_SHAPE),
    (dict(dh=A + 8), lpq.ERR_ALIGN), (dict(dw=A + 4), lpq.ERR_ALIGN), (dict(dloss=A + 1), lpq.ERR_ALIGN)])
def test_loss_backward_refusals(kw, status):
    assert ce_back(**kw) == status


def test_loss_workspace():
    n = ctypes.c_size_t()

    def size(t, v, d, backward, piece=0):
        st = lpq.lib().lpq_linear_ce_workspace(t, v, d, backward, piece, ctypes.byref(n))
        return n.value if st == lpq.OK else -st

    assert size(0, 100, 64, 0) == 0 and size(0, 100, 64, 1) == 0
    # far below the logits' size, and governed by the piece
    t, v, d = 65536, 131072, 4096
    logits = 4 * t * v
    assert size(t, v, d, 0) < logits / 16
    assert size(t, v, d, 1) < logits / 8
    assert size(t, v, d, 1, 1024) < size(t, v, d, 1, 4096)
    assert size(t, v, 60, 1) == -lpq.ERR_SHAPE and size(t, 0, d, 0) == -lpq.ERR_SHAPE and size(t, v, d, 1, 100) == -lpq.ERR_SHAPE
    assert lpq.lib().lpq_linear_ce_workspace(1, 1, 8, 0, 0, None) == lpq.ERR_INVALID_ARG


def mv(fmt=lpq.NVFP4, rows=32, cols=64, codes=A, scales=A, ts=A, layout=lpq.SF_GEMM, colwise=0, x=A, ldx=64, m=1, y=A, fp32=0):
    w = lpq.QView(codes, scales, ts, None, rows, cols, fmt, layout, colwise, 0)
    return lpq.lib().lpq_matvec(ctypes.byref(w), x, ldx, m, y, fp32, None)


@pytest.mark.parametrize("kw,status", [
    (dict(fmt=lpq.BF16), lpq.ERR_UNSUPPORTED), (dict(fmt=lpq.MXFP8), lpq.ERR_UNSUPPORTED), (dict(fmt=lpq.FP8_BLOCK_128x128), lpq.ERR_UNSUPPORTED),
    (dict(colwise=1), lpq.ERR_INVALID_ARG), (dict(layout=2), lpq.ERR_INVALID_ARG), (dict(fp32=3), lpq.ERR_INVALID_ARG),
    (dict(m=-1), lpq.ERR_SHAPE), (dict(rows=-1), lpq.ERR_SHAPE), (dict(cols=48, ldx=48), lpq.ERR_SHAPE), (dict(ldx=56), lpq.ERR_SHAPE),
    (dict(ldx=68), lpq.ERR_SHAPE), (dict(y=None), lpq.ERR_INVALID_ARG), (dict(x=None), lpq.ERR_INVALID_ARG), (dict(codes=None), lpq.ERR_INVALID_ARG),
    (dict(scales=None), lpq.ERR_INVALID_ARG), (dict(ts=None), lpq.ERR_INVALID_ARG), (dict(x=A + 8), lpq.ERR_ALIGN), (dict(y=A + 2), lpq.ERR_ALIGN),
    (dict(codes=A + 4), lpq.ERR_ALIGN), (dict(scales=A + 2), lpq.ERR_ALIGN), (dict(ts=A + 2), lpq.ERR_ALIGN)])
def test_matvec_refusals(kw, status):
    assert mv(**kw) == status


def test_matvec_null_view():
    assert lpq.lib().lpq_matvec(None, A, 64, 1, A, 0, None) == lpq.ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(), dict(fmt=lpq.MXFP4, ts=None), dict(fmt=lpq.NVFP4_2D, layout=lpq.SF_PLAIN), dict(m=0, x=None, y=None),
                                dict(rows=0, y=None, codes=None)])
def test_matvec_accepts(kw):
    if lpq.torch.cuda.is_available():
        pytest.skip("the addresses are not memory")
    assert mv(**kw) in VALID
