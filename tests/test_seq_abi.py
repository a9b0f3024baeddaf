"""The C ABI of the sequence operators: every declared function is exported, the
binding's structs have the header's layout, and bad calls are refused before
anything is queued (no GPU: the placeholder pointers are never touched)."""
import ctypes
import os
import re

import pytest

import convolution_nhwc_conv2d_amd as cn
from convolution_nhwc_conv2d_amd import sequence as sq

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "cnhwc_seq.h")
A = 1 << 28  # placeholder device addresses, far apart


def test_every_declared_function_is_exported():
    text = re.sub(r"/\*.*?\*/", " ", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\bcnhwc_status_t\s+(cnhwc_\w+)\s*\(", text))
    assert names == set(cn.SEQ_EXPORTED)
    for n in names:
        assert hasattr(cn.lib, n), n


def test_constants_and_struct_sizes():
    text = open(HEADER).read()
    assert int(re.search(r"CNHWC_CAUSAL_CONV_MAX_K (\d+)", text).group(1)) == sq.CAUSAL_CONV_MAX_K
    assert int(re.search(r"CNHWC_SCAN_MAX_STATE (\d+)", text).group(1)) == sq.SCAN_MAX_STATE
    assert ctypes.sizeof(sq.LayerNormDesc) == 2 * 4 + 3 * 8 + 4 * 8 + 2 * 4
    assert ctypes.sizeof(sq.CausalConvDesc) == 2 * 4 + 3 * 8 + 2 * 4 + 4 * 8
    assert ctypes.sizeof(sq.ScanDesc) == 2 * 4 + 3 * 8 + 2 * 4 + 12 * 8
    assert ctypes.sizeof(sq.ScanInputs) == 10 * 8 and ctypes.sizeof(sq.ScanGradPointers) == 9 * 8


def _norm(**kw):
    v = dict(dtype=2, w_dtype=2, n=2, l=3, c=64, xs=(192, 64), gs=(192, 64), eps=1e-5)
    v.update(kw)
    return sq._norm_desc(*[v[k] for k in ("dtype", "w_dtype", "n", "l", "c", "xs", "gs", "eps")])


def _conv(**kw):
    v = dict(dtype=1, act=1, n=2, l=3, c=64, k=4, xs=(192, 64), gs=(192, 64))
    v.update(kw)
    return sq._conv_desc(*[v[k] for k in ("dtype", "act", "n", "l", "c", "k", "xs", "gs")])


def _scan(**kw):
    st = (192, 64)
    v = dict(dtype=0, softplus=1, n=2, l=3, d=64, s=16, us=st, ds=st, bs=(48, 16), cs=(48, 16), gs=st, ys=st)
    v.update(kw)
    return sq._scan_desc(*[v[k] for k in ("dtype", "softplus", "n", "l", "d", "s", "us", "ds", "bs", "cs", "gs", "ys")])


BAD = [dict(dtype=3), dict(dtype=-1), dict(n=0), dict(l=0), dict(n=1 << 31), dict(l=-4)]


@pytest.mark.parametrize("bad", BAD + [dict(c=0), dict(xs=(-1, 64)), dict(xs=(1 << 60, 64)), dict(eps=-1.0),
                                       dict(eps=float("nan")), dict(w_dtype=1), dict(gs=(192, -64))], ids=str)
def test_norm_descriptors(bad):
    d, need = _norm(**bad), ctypes.c_uint64()
    assert cn.lib.cnhwc_layer_norm_bwd_workspace(ctypes.byref(d), 1, ctypes.byref(need)) == 1
    assert cn.lib.cnhwc_layer_norm_bwd(ctypes.byref(d), *[A * i for i in range(1, 10)], 1 << 20, None) == 1


@pytest.mark.parametrize("bad", BAD + [dict(c=0), dict(xs=(-1, 64)), dict(act=2), dict(k=0), dict(gs=(192, -64))],
                         ids=str)
def test_conv_descriptors(bad):
    d, need = _conv(**bad), ctypes.c_uint64()
    assert cn.lib.cnhwc_causal_conv_bwd_workspace(ctypes.byref(d), ctypes.byref(need)) == 1


@pytest.mark.parametrize("bad", BAD + [dict(d=0), dict(s=0), dict(softplus=2), dict(us=(-1, 64)), dict(bs=(48, -16)),
                                       dict(ys=(192, -64)), dict(gs=(1 << 61, 64))], ids=str)
def test_scan_descriptors(bad):
    d, need = _scan(**bad), ctypes.c_uint64()
    assert cn.lib.cnhwc_scan_bwd_workspace(ctypes.byref(d), ctypes.byref(need)) == 1


def test_unsupported_sizes():
    need = ctypes.c_uint64()
    for d, f in ((_conv(k=9), cn.lib.cnhwc_causal_conv_bwd_workspace), (_scan(s=65), cn.lib.cnhwc_scan_bwd_workspace),
                 (_conv(l=(1 << 31) - 8), cn.lib.cnhwc_causal_conv_bwd_workspace),
                 (_scan(l=(1 << 31) - 8), cn.lib.cnhwc_scan_bwd_workspace)):
        assert f(ctypes.byref(d), ctypes.byref(need)) == 2
    d = _norm(c=1 << 27, xs=(0, 0), gs=(0, 0))
    assert cn.lib.cnhwc_layer_norm_bwd_workspace(ctypes.byref(d), 1, ctypes.byref(need)) == 2


def test_norm_buffers():
    d = ctypes.byref(_norm())
    f = cn.lib.cnhwc_layer_norm_fwd
    ok = [A, 2 * A, 3 * A, 4 * A, 5 * A, 6 * A]

    def call(**kw):
        v = list(ok)
        for k, p in kw.items():
            v["x w b y mean rstd".split().index(k)] = p
        return f(d, *v, None)
    assert call(x=None) == 1 and call(y=None) == 1 and call(mean=None) == 1 and call(rstd=None) == 1
    assert call(x=A + 1) == 1 and call(mean=5 * A + 2) == 1 and call(w=None) == 1
    assert call(y=A) == 1 and call(y=A + 256) == 1 and call(rstd=5 * A + 4) == 1 and call(mean=4 * A + 64) == 1
    need = ctypes.c_uint64()
    assert cn.lib.cnhwc_layer_norm_bwd_workspace(d, 1, ctypes.byref(need)) == 0 and need.value > 0
    g = cn.lib.cnhwc_layer_norm_bwd
    p = [A * i for i in range(1, 10)]  # dy x mean rstd w dx dw db workspace
    assert g(d, *p, need.value - 1, None) == 5
    assert g(d, *p[:7], None, p[8], need.value, None) == 1      # dw without db
    assert g(d, *p[:8], p[8] + 8, need.value, None) == 1        # workspace off its alignment
    assert g(d, *p[:5], p[0], *p[6:], need.value, None) == 1    # dx on dy
    assert g(d, *p[:4], None, *p[5:], need.value, None) == 1    # dw without w


def test_conv_buffers():
    d, one = ctypes.byref(_conv()), ctypes.byref(_conv(l=1))
    f, s = cn.lib.cnhwc_causal_conv_fwd, cn.lib.cnhwc_causal_conv_step
    p = [A * i for i in range(1, 8)]  # x w bias state lengths y state_out
    for i in (0, 1, 5):
        assert f(d, *p[:i], None, *p[i + 1:], None) == 1
    assert f(d, *p[:4], p[4] + 2, *p[5:], None) == 1            # lengths off their alignment
    assert f(d, *p[:5], p[0] + 128, p[6], None) == 1            # y inside x
    assert f(d, *p[:6], p[3], None) == 1                        # the new state on the old one
    q = [A * i for i in range(1, 7)]  # x state w bias y state_out
    assert s(d, *q, None) == 1                                  # more than one position
    for i in (0, 1, 2, 4, 5):
        assert s(one, *q[:i], None, *q[i + 1:], None) == 1
    assert s(one, *q[:5], q[1] + 64, None) == 1                 # states that overlap in part
    need = ctypes.c_uint64()
    assert cn.lib.cnhwc_causal_conv_bwd_workspace(d, ctypes.byref(need)) == 0
    g = cn.lib.cnhwc_causal_conv_bwd
    r = [A * i for i in range(1, 13)]  # dy dstate_out x w bias state lengths dx dw dbias dstate workspace
    assert g(d, *r, need.value - 1, None) == 5
    assert g(d, *r[:9], None, *r[10:], need.value, None) == 1   # bias without its gradient
    assert g(d, *r[:7], r[2], *r[8:], need.value, None) == 1    # dx on x


def _ins(**kw):
    v = {f: A * (i + 1) for i, (f, _) in enumerate(sq.ScanInputs._fields_)}
    v.update(kw)
    return ctypes.byref(sq.ScanInputs(**v))


def _grads(**kw):
    v = {f: A * (i + 21) for i, (f, _) in enumerate(sq.ScanGradPointers._fields_)}
    v.update(kw)
    return ctypes.byref(sq.ScanGradPointers(**v))


def test_scan_buffers():
    d, one = ctypes.byref(_scan()), ctypes.byref(_scan(l=1))
    f, s, g = cn.lib.cnhwc_scan_fwd, cn.lib.cnhwc_scan_step, cn.lib.cnhwc_scan_bwd
    Y, S, W = 40 * A, 41 * A, 42 * A
    for name in ("u", "delta", "a", "b", "c"):
        assert f(d, _ins(**{name: None}), Y, S, W, 1 << 27, None) == 1
        assert f(d, _ins(**{name: A + 1}), Y, S, W, 1 << 27, None) == 1
    assert f(d, None, Y, S, W, 1 << 27, None) == 1
    assert f(d, _ins(), None, S, W, 1 << 27, None) == 1
    assert f(d, _ins(), A, S, W, 1 << 27, None) == 1            # y on u
    assert f(d, _ins(), Y, 9 * A, W, 1 << 27, None) == 1        # the new state on the old one
    assert s(d, _ins(lengths=None), Y, S, None) == 1            # more than one position
    assert s(one, _ins(), Y, S, None) == 1                      # lengths
    assert s(one, _ins(lengths=None, state=None), Y, S, None) == 1
    assert s(one, _ins(lengths=None), Y, None, None) == 1
    assert s(one, _ins(lengths=None), Y, 9 * A + 64, None) == 1  # states that overlap in part
    need = ctypes.c_uint64()
    assert cn.lib.cnhwc_scan_bwd_workspace(d, ctypes.byref(need)) == 0 and need.value > 0
    assert g(d, _ins(), Y, S, _grads(), W, need.value - 1, None) == 5
    for name in ("u", "delta", "a", "b", "c", "skip", "gate", "delta_bias"):
        assert g(d, _ins(), Y, S, _grads(**{name: None}), W, need.value, None) == 1
    for name in ("skip", "gate", "delta_bias"):
        assert g(d, _ins(**{name: None}), Y, S, _grads(), W, need.value, None) == 1
    assert g(d, _ins(), Y, S, _grads(u=A), W, need.value, None) == 1
    assert g(d, _ins(), Y, S, _grads(), W + 4, need.value, None) == 1
