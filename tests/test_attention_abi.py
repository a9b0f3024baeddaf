"""The C ABI of the root-mean-square norm, rotary positions and linear attention:
struct layouts, and refusals before anything is queued (no GPU: the placeholder
pointers are never touched)."""
import ctypes
import os
import re

import pytest

import convolution_nhwc_conv2d_amd as cn
from convolution_nhwc_conv2d_amd import sequence as sq

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "cnhwc_seq.h")
A = 1 << 28  # placeholder device addresses, far apart
INVALID, UNSUPPORTED, SMALL = 1, 2, 5


def test_constants_and_struct_sizes():
    text = open(HEADER).read()
    assert int(re.search(r"CNHWC_LINEAR_ATTENTION_MAX_DIM (\d+)", text).group(1)) == sq.LINEAR_ATTENTION_MAX_DIM
    assert ctypes.sizeof(sq.RmsNormDesc) == 2 * 4 + 3 * 8 + 6 * 8 + 2 * 4
    assert ctypes.sizeof(sq.RotaryDesc) == 2 * 4 + 3 * 8 + 2 * 4 + 8 * 8 + 8 + 2 * 4 + 8
    assert ctypes.sizeof(sq.LinearAttentionDesc) == 2 * 4 + 3 * 8 + 2 * 4 + 12 * 8 + 2 * 4
    assert ctypes.sizeof(sq.LinearAttentionInputs) == 6 * 8 and ctypes.sizeof(sq.LinearAttentionGradPointers) == 5 * 8


def _rms(**kw):
    v = dict(dtype=2, w_dtype=2, n=2, l=3, c=64, xs=(192, 64), rs=(192, 64), gs=(192, 64), eps=1e-6, group=0)
    v.update(kw)
    return ctypes.byref(sq._rms_desc(*[v[k] for k in ("dtype", "w_dtype", "n", "l", "c", "xs", "rs", "gs", "eps",
                                                      "group")]))


def _rot(**kw):
    d = sq.RotaryDesc(dtype=2, n=2, l=3, h=4, d=64, r=32, scale=1.0)
    strides = dict(xs=(768, 256, 64), os=(768, 256, 64), ps=(3, 1))
    strides.update({k: kw.pop(k) for k in list(kw) if k in strides})
    d.x_stride[:], d.out_stride[:], d.position_stride[:] = strides["xs"], strides["os"], strides["ps"]
    for k, v in kw.items():
        setattr(d, k, v)
    return ctypes.byref(d)


def _att(**kw):
    wide = (768, 256, 64)
    v = dict(dtype=2, n=2, l=3, h=4, dk=64, dv=64, qs=wide, ks=wide, vs=wide, gs=wide)
    more = {k: kw.pop(k) for k in ("reserved", "reserved2") if k in kw}
    v.update(kw)
    d = sq._attention_desc(*[v[k] for k in ("dtype", "n", "l", "h", "dk", "dv", "qs", "ks", "vs", "gs")])
    for k, x in more.items():
        setattr(d, k, x)
    return ctypes.byref(d)


SIZES = [dict(dtype=3), dict(dtype=-1), dict(n=0), dict(l=0), dict(n=1 << 31), dict(l=-4)]


@pytest.mark.parametrize("bad", SIZES + [dict(c=0), dict(xs=(-1, 64)), dict(xs=(1 << 60, 64)), dict(eps=-1.0),
                                         dict(eps=float("nan")), dict(w_dtype=1), dict(rs=(192, -64)), dict(group=32)],
                         ids=str)
def test_rms_descriptors(bad):
    p = [A * i for i in range(1, 9)]
    f, q = cn.lib.cnhwc_rms_norm_fwd, cn.lib.cnhwc_rms_norm_fwd_q8
    assert f(_rms(**bad), *p[:6], None) == INVALID
    if "group" not in bad:
        assert q(_rms(**bad), *p[:7], None) == INVALID
    if "rs" not in bad:
        need = ctypes.c_uint64()
        assert cn.lib.cnhwc_rms_norm_bwd_workspace(_rms(**bad), 1, ctypes.byref(need)) == INVALID


def test_rms_groups():
    p = [A * i for i in range(1, 9)]
    q = cn.lib.cnhwc_rms_norm_fwd_q8
    for group in (-32, 48, 128):  # not a divisor of 64
        assert q(_rms(group=group), *p[:7], None) == INVALID
    for group in (1, 16, 64 * 4):
        assert q(_rms(c=1024, xs=(3 << 10, 1 << 10), rs=(3 << 10, 1 << 10), group=group), *p[:7], None) == UNSUPPORTED
    big = _rms(c=1 << 27, xs=(0, 0), gs=(0, 0))
    assert cn.lib.cnhwc_rms_norm_bwd_workspace(big, 1, ctypes.byref(ctypes.c_uint64())) == UNSUPPORTED


def test_rms_buffers():
    names = "x residual w y sum rstd".split()
    ok = [A * i for i in range(1, 7)]

    def call(desc=None, **kw):
        v = list(ok)
        for k, p in kw.items():
            v[names.index(k)] = p
        return cn.lib.cnhwc_rms_norm_fwd(desc or _rms(), *v, None)
    assert call(x=None) == INVALID and call(y=None) == INVALID and call(residual=None) == INVALID
    assert call(x=A + 1) == INVALID and call(rstd=6 * A + 2) == INVALID
    assert call(y=A) == INVALID and call(sum=A) == INVALID and call(sum=2 * A + 64) == INVALID
    assert call(y=5 * A) == INVALID and call(rstd=4 * A) == INVALID and call(y=2 * A) == INVALID
    assert call(sum=2 * A, desc=_rms(rs=(0, 64))) == INVALID and call(sum=2 * A, desc=_rms(rs=(192, 128))) == INVALID
    q = [A * i for i in range(1, 8)]  # x residual w q scale sum rstd
    for i in (0, 3, 4):
        assert cn.lib.cnhwc_rms_norm_fwd_q8(_rms(), *q[:i], None, *q[i + 1:], None) == INVALID
    assert cn.lib.cnhwc_rms_norm_fwd_q8(_rms(), *q[:4], q[3], *q[5:], None) == INVALID  # scale on q
    need = ctypes.c_uint64()
    assert cn.lib.cnhwc_rms_norm_bwd_workspace(_rms(), 1, ctypes.byref(need)) == 0 and need.value > 0
    g = cn.lib.cnhwc_rms_norm_bwd
    p = [A * i for i in range(1, 9)]  # dy dsum x rstd w dx dw workspace
    assert g(_rms(), *p, need.value - 1, None) == SMALL
    for i in (0, 2, 3, 5):
        assert g(_rms(), *p[:i], None, *p[i + 1:], need.value, None) == INVALID
    assert g(_rms(), *p[:4], None, *p[5:], need.value, None) == INVALID             # dw without w
    assert g(_rms(), *p[:7], p[7] + 8, need.value, None) == INVALID                 # workspace off its alignment
    assert g(_rms(), *p[:5], p[1], *p[6:], need.value, None) == INVALID             # dx on dsum


@pytest.mark.parametrize("bad", SIZES + [dict(h=0), dict(d=0), dict(r=-2), dict(r=31), dict(r=66), dict(interleaved=2),
                                         dict(inverse=-1), dict(xs=(-1, 256, 64)), dict(os=(768, 256, -64)),
                                         dict(ps=(-3, 1)), dict(offset=1 << 41), dict(offset=-(1 << 41)),
                                         dict(reserved=1), dict(xs=(768, 1 << 60, 64)),
                                         dict(os=(768, 256, 0)), dict(os=(768, 192, 64)), dict(os=(0, 256, 64))],
                         ids=str)
def test_rotary_descriptors(bad):
    assert cn.lib.cnhwc_rotary(_rot(**bad), A, 2 * A, 3 * A, 4 * A, None) == INVALID


def test_rotary_buffers():
    f = cn.lib.cnhwc_rotary
    for p in ((None, 2 * A, 3 * A, 4 * A), (A, None, 3 * A, 4 * A), (A, 2 * A, 3 * A, None), (A + 1, 2 * A, 3 * A, 4 * A),
              (A, 2 * A + 4, 3 * A, 4 * A), (A, 2 * A, 3 * A + 2, 4 * A), (A, 2 * A, 3 * A, A + 64),
              (A, 2 * A, 3 * A, 2 * A), (A, 2 * A, 3 * A, 3 * A)):
        assert f(_rot(), *p, None) == INVALID, p
    assert f(_rot(xs=(768, 256, 128)), A, 2 * A, None, A, None) == INVALID  # in place with other strides


@pytest.mark.parametrize("bad", SIZES + [dict(h=0), dict(dk=0), dict(dv=-1), dict(qs=(-1, 256, 64)), dict(reserved=1),
                                         dict(ks=(768, -256, 64)), dict(vs=(768, 256, -1)), dict(gs=(768, 256, -1)),
                                         dict(qs=(1 << 60, 256, 64)), dict(reserved2=1)], ids=str)
def test_attention_descriptors(bad):
    need = ctypes.c_uint64()
    assert cn.lib.cnhwc_linear_attention_bwd_workspace(_att(**bad), 1, ctypes.byref(need)) == INVALID
    if "gs" not in bad:
        assert cn.lib.cnhwc_linear_attention_fwd_workspace(_att(**bad), ctypes.byref(need)) == INVALID


def test_attention_sizes():
    need = ctypes.c_uint64()
    for bad in (dict(dk=257), dict(dv=300), dict(n=1 << 20, h=1 << 20, qs=(0, 0, 0), ks=(0, 0, 0), vs=(0, 0, 0)),
                dict(l=(1 << 31) - 1, qs=(0, 0, 0), ks=(0, 0, 0), vs=(0, 0, 0))):
        assert cn.lib.cnhwc_linear_attention_fwd_workspace(_att(**bad), ctypes.byref(need)) == UNSUPPORTED
    assert cn.lib.cnhwc_linear_attention_fwd_workspace(_att(), None) == INVALID


def _ins(**kw):
    v = {f: A * (i + 1) for i, (f, _) in enumerate(sq.LinearAttentionInputs._fields_)}
    v.update(kw)
    return ctypes.byref(sq.LinearAttentionInputs(**v))


def _grads(**kw):
    v = {f: A * (i + 21) for i, (f, _) in enumerate(sq.LinearAttentionGradPointers._fields_)}
    v.update(kw)
    return ctypes.byref(sq.LinearAttentionGradPointers(**v))


def test_attention_buffers():
    f, s, g = cn.lib.cnhwc_linear_attention_fwd, cn.lib.cnhwc_linear_attention_step, cn.lib.cnhwc_linear_attention_bwd
    Y, S, W, big = 40 * A, 41 * A, 42 * A, 1 << 27
    for name in ("q", "k", "v", "log_decay"):
        assert f(_att(), _ins(**{name: None}), Y, S, W, big, None) == INVALID
        assert f(_att(), _ins(**{name: A + 1}), Y, S, W, big, None) == INVALID
    assert f(_att(), None, Y, S, W, big, None) == INVALID
    assert f(_att(), _ins(), None, S, W, big, None) == INVALID
    assert f(_att(), _ins(), A, S, W, big, None) == INVALID             # y on q
    assert f(_att(), _ins(), Y, 5 * A, W, big, None) == INVALID         # the new state on the old one
    one = dict(l=1)
    assert s(_att(), _ins(lengths=None), Y, S, None) == INVALID         # more than one position
    assert s(_att(**one), _ins(), Y, S, None) == INVALID                # lengths
    assert s(_att(**one), _ins(lengths=None, state=None), Y, S, None) == INVALID
    assert s(_att(**one), _ins(lengths=None), Y, None, None) == INVALID
    assert s(_att(**one), _ins(lengths=None), Y, 5 * A + 64, None) == INVALID  # states that overlap in part
    need = ctypes.c_uint64()
    assert cn.lib.cnhwc_linear_attention_bwd_workspace(_att(), 1, ctypes.byref(need)) == 0 and need.value > 0
    assert g(_att(), _ins(), Y, S, _grads(), W, need.value - 1, None) == SMALL
    assert g(_att(), _ins(), Y, S, None, W, need.value, None) == INVALID
    assert g(_att(), _ins(), None, S, _grads(), W, need.value, None) == INVALID
    for name in ("q", "k", "v"):
        assert g(_att(), _ins(), Y, S, _grads(**{name: None}), W, need.value, None) == INVALID
    assert g(_att(), _ins(), Y, S, _grads(q=A), W, need.value, None) == INVALID
    assert g(_att(), _ins(), Y, S, _grads(), W + 4, need.value, None) == INVALID
