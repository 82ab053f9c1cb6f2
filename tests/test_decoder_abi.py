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
    (dict(v=(1 << 31) + 1, ld=1 << 32, ldo=1 << 32), lpq.ERR_SHAPE), (dict(ld=99), lpq.ERR_SHAPE), (dict(ldo=99), lpq.ERR_SHAPE), (dict(x=None), lpq.ERR_INVALID_ARG),
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
