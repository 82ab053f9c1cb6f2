"""Argument checks of the head norm, adapter, expert and logit entry points: all
of it is decided on the host, without a GPU."""
import ctypes
import math

import pytest

from precision_transformer_gemms_gb300 import lpq

A = 1 << 20  # an aligned address that is never read
VALID = (lpq.OK, lpq.ERR_ARCH, lpq.ERR_CUDA)  # arguments accepted: stops at the device check here
on_cpu = pytest.mark.skipif(lpq.torch.cuda.is_available(), reason="the addresses are not memory")


def freqs(n, bad=None):
    return (ctypes.c_double * max(1, n))(*[bad if i == 1 and bad is not None else 0.5 for i in range(n)])


def qk(x=A, ldx=512, t=0, rows=4, hq=2, hk=1, d=64, qw=A, kw=A, wt=0, pos=A, f=freqs(256), rot=64, inter=0, eps=1e-6, y=A, ldy=512):
    return lpq.lib().lpq_qk_norm_rope(x, ldx, t, rows, hq, hk, d, qw, kw, wt, pos, f, rot, inter, eps, y, ldy, None)


def qk_back(dy=A, lddy=512, x=A, ldx=512, t=0, rows=4, hq=2, hk=1, d=64, qw=A, kw=A, wt=0, pos=A, f=freqs(256), rot=64, inter=0, eps=1e-6,
            y=A, ldy=512, dq=A, dk=A, ws=A, wsb=1 << 30):
    return lpq.lib().lpq_qk_norm_rope_backward(dy, lddy, x, ldx, t, rows, hq, hk, d, qw, kw, wt, pos, f, rot, inter, eps, y, ldy, dq, dk, ws,
                                               wsb, None)


@pytest.mark.parametrize("call", [qk, qk_back])
@pytest.mark.parametrize("kw,status", [
    (dict(t=2), lpq.ERR_INVALID_ARG), (dict(wt=5), lpq.ERR_INVALID_ARG), (dict(inter=2), lpq.ERR_INVALID_ARG), (dict(eps=-1.0), lpq.ERR_INVALID_ARG),
    (dict(eps=math.nan), lpq.ERR_INVALID_ARG), (dict(d=0, rot=0), lpq.ERR_SHAPE), (dict(d=63), lpq.ERR_SHAPE), (dict(d=514, ldx=9999, ldy=9999), lpq.ERR_SHAPE),
    (dict(rot=66), lpq.ERR_SHAPE), (dict(rot=31), lpq.ERR_SHAPE), (dict(rot=-2), lpq.ERR_SHAPE), (dict(rows=-1), lpq.ERR_SHAPE),
    (dict(hq=-1), lpq.ERR_SHAPE), (dict(hk=-3), lpq.ERR_SHAPE), (dict(hq=1 << 21, ldx=1 << 40, ldy=1 << 40), lpq.ERR_SHAPE), (dict(ldx=191), lpq.ERR_SHAPE),
    (dict(ldy=64), lpq.ERR_SHAPE), (dict(x=None), lpq.ERR_INVALID_ARG), (dict(y=None), lpq.ERR_INVALID_ARG), (dict(pos=None), lpq.ERR_INVALID_ARG),
    (dict(pos=A + 4), lpq.ERR_ALIGN), (dict(f=None), lpq.ERR_INVALID_ARG), (dict(f=freqs(256, math.inf)), lpq.ERR_INVALID_ARG),
    (dict(f=freqs(256, math.nan)), lpq.ERR_INVALID_ARG), (dict(x=A + 1), lpq.ERR_ALIGN), (dict(t=1, y=A + 2), lpq.ERR_ALIGN), (dict(qw=A + 1), lpq.ERR_ALIGN),
    (dict(wt=1, kw=A + 2), lpq.ERR_ALIGN), (dict(ldx=320), lpq.ERR_SHAPE)])
def test_head_norm_refusals(call, kw, status):
    assert call(**kw) == status
    assert lpq.last_error()


@pytest.mark.parametrize("kw,status", [
    (dict(dy=None), lpq.ERR_INVALID_ARG), (dict(lddy=100), lpq.ERR_SHAPE), (dict(dy=A + 1), lpq.ERR_ALIGN), (dict(dq=A + 2), lpq.ERR_ALIGN),
    (dict(dk=A + 1), lpq.ERR_ALIGN), (dict(ws=None), lpq.ERR_INVALID_ARG), (dict(wsb=64), lpq.ERR_INVALID_ARG), (dict(ws=A + 8), lpq.ERR_ALIGN),
    (dict(lddy=400), lpq.ERR_SHAPE)])
def test_head_norm_backward_refusals(kw, status):
    assert qk_back(**kw) == status


@on_cpu
@pytest.mark.parametrize("kw", [dict(), dict(qw=None, kw=None), dict(rows=0, x=None, y=None, pos=None), dict(hq=0, hk=0, x=None, y=None, pos=None, ldx=0, ldy=0),
                                dict(rot=0, f=None), dict(d=2, rot=2), dict(d=512, rot=512, ldx=1536, ldy=1536), dict(inter=1, x=A + 2, ldx=777, y=A + 6, ldy=555)])
def test_head_norm_accepts(kw):
    assert qk(**kw) in VALID


@on_cpu
def test_head_norm_backward_accepts():
    assert qk_back() in VALID
    assert qk_back(dq=None, dk=None, ws=None, wsb=0) in VALID
    assert qk_back(rows=0, dy=None, x=None, y=None, pos=None, ws=None, wsb=0) in VALID


def test_head_norm_workspace():
    n = ctypes.c_size_t(7)
    size = lambda r, d: (lpq.lib().lpq_qk_norm_rope_workspace(r, d, ctypes.byref(n)), n.value)
    assert size(0, 128) == (0, 0)
    assert size(5, 128)[0] == 0 and 0 < size(10 ** 9, 512)[1] <= 4 << 20
    assert size(-1, 128)[0] == lpq.ERR_SHAPE and size(1, 514)[0] == lpq.ERR_SHAPE
    assert lpq.lib().lpq_qk_norm_rope_workspace(1, 64, None) == lpq.ERR_INVALID_ARG


def adjust(x=A, ld=100, t=1, rows=3, v=100, out=A, ldo=100, null=False, **kw):
    c = dict(history=A, ld_history=8, max_len=8, lengths=A, prompt=A, repetition=A, frequency=A, presence=A, bias_offsets=A, bias_words=A, bias_values=A,
             bias_count=4, allowed=A, ld_allowed=4)
    c.update(kw)
    c = lpq.LogitControls(*[c[n] for n, _ in lpq.LogitControls._fields_])
    return lpq.lib().lpq_adjust_logits(x, ld, t, rows, v, None if null else ctypes.addressof(c), out, ldo, None)


@pytest.mark.parametrize("kw,status", [
    (dict(null=True), lpq.ERR_INVALID_ARG), (dict(t=2), lpq.ERR_INVALID_ARG), (dict(rows=-1), lpq.ERR_SHAPE), (dict(v=-1), lpq.ERR_SHAPE),
    (dict(v=(1 << 30) + 1, ld=1 << 32, ldo=1 << 32), lpq.ERR_SHAPE), (dict(ld=99), lpq.ERR_SHAPE), (dict(ldo=99), lpq.ERR_SHAPE), (dict(x=None), lpq.ERR_INVALID_ARG),
    (dict(out=None), lpq.ERR_INVALID_ARG), (dict(x=A + 2), lpq.ERR_ALIGN), (dict(t=0, out=A + 1), lpq.ERR_ALIGN), (dict(ld=104), lpq.ERR_SHAPE),
    (dict(max_len=9), lpq.ERR_SHAPE), (dict(max_len=-1), lpq.ERR_SHAPE), (dict(lengths=None), lpq.ERR_INVALID_ARG),
    (dict(history=None, lengths=None, prompt=None), lpq.ERR_INVALID_ARG), (dict(bias_offsets=None), lpq.ERR_INVALID_ARG),
    (dict(bias_values=None), lpq.ERR_INVALID_ARG), (dict(bias_count=-1), lpq.ERR_SHAPE), (dict(ld_allowed=3), lpq.ERR_SHAPE), (dict(history=A + 4), lpq.ERR_ALIGN),
    (dict(lengths=A + 4), lpq.ERR_ALIGN), (dict(bias_words=A + 1), lpq.ERR_ALIGN), (dict(repetition=A + 2), lpq.ERR_ALIGN), (dict(allowed=A + 2), lpq.ERR_ALIGN)])
def test_logits_refusals(kw, status):
    assert adjust(**kw) == status
    assert lpq.last_error()


@on_cpu
@pytest.mark.parametrize("kw", [dict(), dict(history=None, lengths=None, prompt=None, repetition=None, frequency=None, presence=None), dict(prompt=None),
                                dict(bias_words=None, bias_offsets=None, bias_values=None), dict(allowed=None, ld_allowed=0), dict(rows=0, x=None, out=None),
                                dict(v=0, ld=0, ldo=0, x=None, out=None), dict(out=A + 4, ldo=117)])
def test_logits_accepts(kw):
    assert adjust(**kw) in VALID


def adapted(a=A, b=A, scale=A, count=2, rank=16, index=A, ws=A, wsb=1 << 20, null=False, fmt=lpq.NVFP4, rows=32, cols=64, x=A, ldx=64, m=1, y=A, fp32=0):
    w = lpq.QView(A, A, A, None, rows, cols, fmt, lpq.SF_GEMM, 0, 0)
    ad = lpq.AdaptersC(a, b, scale, count, rank)
    return lpq.lib().lpq_matvec_adapted(ctypes.byref(w), x, ldx, m, y, fp32, None if null else ctypes.byref(ad), index, ws, wsb, None)


@pytest.mark.parametrize("kw,status", [
    (dict(null=True), lpq.ERR_INVALID_ARG), (dict(rank=0), lpq.ERR_SHAPE), (dict(rank=12), lpq.ERR_SHAPE), (dict(rank=264), lpq.ERR_SHAPE),
    (dict(rank=-8), lpq.ERR_SHAPE), (dict(count=-1), lpq.ERR_SHAPE), (dict(a=None), lpq.ERR_INVALID_ARG), (dict(b=None), lpq.ERR_INVALID_ARG),
    (dict(index=None), lpq.ERR_INVALID_ARG), (dict(a=A + 8), lpq.ERR_ALIGN), (dict(b=A + 2), lpq.ERR_ALIGN), (dict(scale=A + 2), lpq.ERR_ALIGN),
    (dict(index=A + 4), lpq.ERR_ALIGN), (dict(ws=None), lpq.ERR_INVALID_ARG), (dict(wsb=63), lpq.ERR_INVALID_ARG), (dict(ws=A + 8), lpq.ERR_ALIGN),
    (dict(fmt=lpq.BF16), lpq.ERR_UNSUPPORTED), (dict(m=-1), lpq.ERR_SHAPE), (dict(y=None), lpq.ERR_INVALID_ARG), (dict(ldx=56), lpq.ERR_SHAPE)])
def test_adapted_refusals(kw, status):
    assert adapted(**kw) == status


@on_cpu
@pytest.mark.parametrize("kw", [dict(), dict(scale=None), dict(count=0, a=None, b=None, index=None, ws=None, wsb=0), dict(m=0, ws=None, wsb=0, x=None, y=None, index=None)])
def test_adapted_accepts(kw):
    assert adapted(**kw) in VALID


def test_adapted_workspace():
    n = ctypes.c_size_t(7)
    assert lpq.lib().lpq_matvec_adapted_workspace(3, 16, ctypes.byref(n)) == 0 and n.value == 3 * 16 * 4
    assert lpq.lib().lpq_matvec_adapted_workspace(-1, 16, ctypes.byref(n)) == lpq.ERR_SHAPE
    assert lpq.lib().lpq_matvec_adapted_workspace(1, 16, None) == lpq.ERR_INVALID_ARG


def route(x=A, ldx=64, w=A, ldw=64, m=2, d=64, e=8, k=2, renormalize=1, ids=A, probs=A):
    return lpq.lib().lpq_moe_route(x, ldx, w, ldw, m, d, e, k, renormalize, ids, probs, None)


@pytest.mark.parametrize("kw,status", [
    (dict(renormalize=2), lpq.ERR_INVALID_ARG), (dict(m=-1), lpq.ERR_SHAPE), (dict(d=0), lpq.ERR_SHAPE), (dict(d=60), lpq.ERR_SHAPE), (dict(d=65544, ldx=65544, ldw=65544), lpq.ERR_SHAPE), (dict(e=0), lpq.ERR_SHAPE),
    (dict(e=1025), lpq.ERR_SHAPE), (dict(k=0), lpq.ERR_SHAPE), (dict(k=9), lpq.ERR_SHAPE), (dict(e=64, k=33), lpq.ERR_SHAPE), (dict(ldx=56), lpq.ERR_SHAPE),
    (dict(ldw=68), lpq.ERR_SHAPE), (dict(x=None), lpq.ERR_INVALID_ARG), (dict(w=None), lpq.ERR_INVALID_ARG), (dict(ids=None), lpq.ERR_INVALID_ARG),
    (dict(probs=None), lpq.ERR_INVALID_ARG), (dict(x=A + 8), lpq.ERR_ALIGN), (dict(w=A + 2), lpq.ERR_ALIGN), (dict(ids=A + 4), lpq.ERR_ALIGN),
    (dict(probs=A + 2), lpq.ERR_ALIGN)])
def test_route_refusals(kw, status):
    assert route(**kw) == status


@on_cpu
@pytest.mark.parametrize("kw", [dict(), dict(m=0, x=None, ids=None, probs=None), dict(e=1024, k=32), dict(e=1, k=1)])
def test_route_accepts(kw):
    assert route(**kw) in VALID


def moe(fmt=lpq.NVFP4, fmt2=None, layout=lpq.SF_GEMM, colwise=0, d=64, f=96, e=4, rows=None, rows2=None, codes=A, scales=A, ts=A, x=A, ldx=64, m=2, ids=A, probs=A, k=2,
        y=A, ws=A, wsb=1 << 30, null=False):
    up = lpq.QView(codes, scales, ts, None, e * 2 * f if rows is None else rows, d, fmt, layout, colwise, 0)
    down = lpq.QView(codes, scales, ts, None, e * d if rows2 is None else rows2, f, fmt if fmt2 is None else fmt2, layout, colwise, 0)
    return lpq.lib().lpq_moe(None if null else ctypes.addressof(up), ctypes.addressof(down), e, x, ldx, m, ids, probs, k, y, ws, wsb, None)


@pytest.mark.parametrize("kw,status", [
    (dict(null=True), lpq.ERR_INVALID_ARG), (dict(fmt=lpq.MXFP8), lpq.ERR_UNSUPPORTED), (dict(fmt2=lpq.BF16), lpq.ERR_UNSUPPORTED), (dict(layout=lpq.SF_PLAIN), lpq.ERR_UNSUPPORTED),
    (dict(layout=3), lpq.ERR_UNSUPPORTED), (dict(colwise=1), lpq.ERR_INVALID_ARG), (dict(d=48, ldx=48), lpq.ERR_SHAPE), (dict(f=40), lpq.ERR_SHAPE), (dict(f=0), lpq.ERR_SHAPE),
    (dict(d=65568, ldx=65568), lpq.ERR_SHAPE), (dict(e=0), lpq.ERR_SHAPE), (dict(e=1025), lpq.ERR_SHAPE), (dict(rows=700), lpq.ERR_SHAPE), (dict(rows2=128), lpq.ERR_SHAPE),
    (dict(codes=None), lpq.ERR_INVALID_ARG), (dict(scales=None), lpq.ERR_INVALID_ARG), (dict(ts=None), lpq.ERR_INVALID_ARG), (dict(codes=A + 8), lpq.ERR_ALIGN),
    (dict(scales=A + 4), lpq.ERR_ALIGN), (dict(ts=A + 2), lpq.ERR_ALIGN), (dict(x=None), lpq.ERR_INVALID_ARG), (dict(x=A + 8), lpq.ERR_ALIGN), (dict(ldx=56), lpq.ERR_SHAPE),
    (dict(ldx=68), lpq.ERR_SHAPE), (dict(m=-1), lpq.ERR_SHAPE), (dict(k=-1), lpq.ERR_SHAPE), (dict(k=33), lpq.ERR_SHAPE), (dict(ids=None), lpq.ERR_INVALID_ARG),
    (dict(probs=None), lpq.ERR_INVALID_ARG), (dict(ids=A + 4), lpq.ERR_ALIGN), (dict(probs=A + 2), lpq.ERR_ALIGN), (dict(y=None), lpq.ERR_INVALID_ARG), (dict(y=A + 1), lpq.ERR_ALIGN),
    (dict(ws=None), lpq.ERR_INVALID_ARG), (dict(wsb=100), lpq.ERR_INVALID_ARG), (dict(ws=A + 8), lpq.ERR_ALIGN)])
def test_moe_refusals(kw, status):
    assert moe(**kw) == status
    assert lpq.last_error()


@on_cpu
@pytest.mark.parametrize("kw", [dict(), dict(fmt=lpq.MXFP4, fmt2=lpq.NVFP4_2D), dict(fmt=lpq.MXFP4, ts=None), dict(k=0, ids=None, probs=None), dict(m=0, x=None, y=None, ids=None, probs=None, ws=None, wsb=0)])
def test_moe_accepts(kw):
    assert moe(**kw) in VALID


def test_moe_workspace():
    n = ctypes.c_size_t(7)
    size = lambda *a: (lpq.lib().lpq_moe_workspace(*a, ctypes.byref(n)), n.value)
    assert size(8, 8, 4096, 1536)[1] >= 64 * (4096 + 1536) * 4
    assert size(100000, 8, 4096, 1536)[1] < 16 << 20  # the tokens of one launch
    assert size(1, 1, 40, 32)[0] == lpq.ERR_SHAPE and size(1, 33, 32, 32)[0] == lpq.ERR_SHAPE and size(-1, 1, 32, 32)[0] == lpq.ERR_SHAPE
    assert lpq.lib().lpq_moe_workspace(1, 1, 32, 32, None) == lpq.ERR_INVALID_ARG
