"""Sequence operators: layer norm, the short causal convolution and the
selective state space scan -- the binding of ``include/cnhwc_seq.h``.

    layer_norm(x, weight, bias, eps)            layer_norm_backward(dy, x, mean, rstd, weight)
    causal_conv1d(x, w, bias)                   causal_conv1d_backward(dy, x, w, bias)
                                                causal_conv1d_step(x, state, w, bias)
    selective_scan(u, delta, a, b, c)           selective_scan_backward(dy, u, delta, a, b, c)
                                                selective_scan_step(u, delta, a, b, c, state)

Layouts: sequences are channels-last [N, L, C] as for conv1d; a single token is
[N, C].  Inputs need a channel stride of 1 and may otherwise be strided, so the
parts of a projection's rows (``xz[..., :c]``) go in without a copy; parameters,
states, outputs and gradients are dense.  Activations are float32, float16 or
bfloat16; statistics, states and sums are held in float32.

``lengths`` (int32, [N], on the GPU): valid leading positions of each sequence.
Positions past them are never read; outputs and gradients there are 0, and a
state is the one after the last valid position.

The calls launch on the current stream, never synchronise, and allocate only
what they return and their workspace; ``out=`` and ``workspace=`` take both
from the caller.  Nothing is recorded for autograd: the backward functions are
called by the caller, with the forward pass's inputs.

Wrong tensors raise TypeError or ValueError, what the library refuses
CnhwcError.  The checks and calls themselves are compiled (``_seq``, from
csrc/seq_torch.cpp): a single token's kernel takes less time than they would in
Python.
"""
import collections
import ctypes

import torch  # noqa: F401  (before the extension, which uses its libraries)

from . import _DTYPE_CODE, LIB_PATH, CnhwcError, lib

try:
    from . import _seq
except ImportError as e:
    raise ImportError(f"the torch extension beside {LIB_PATH} is not built or does not load ({e}); run "
                      "`python convolution_nhwc_conv2d_amd/build.py`") from e

_seq.set_error(CnhwcError)

_i32, _i64, _f32, _vp, _u64 = ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_void_p, ctypes.c_uint64
_P = ctypes.POINTER

CAUSAL_CONV_MAX_K = 8
SCAN_MAX_STATE = 64

ACTIVATIONS = {None: 0, "silu": 1}


class LayerNormDesc(ctypes.Structure):
    _fields_ = [("dtype", _i32), ("w_dtype", _i32), ("n", _i64), ("l", _i64), ("c", _i64), ("x_stride", _i64 * 2),
                ("dy_stride", _i64 * 2), ("eps", _f32), ("reserved", _i32)]


class CausalConvDesc(ctypes.Structure):
    _fields_ = [("dtype", _i32), ("activation", _i32), ("n", _i64), ("l", _i64), ("c", _i64), ("k", _i32),
                ("reserved", _i32), ("x_stride", _i64 * 2), ("dy_stride", _i64 * 2)]


class ScanDesc(ctypes.Structure):
    _fields_ = [("dtype", _i32), ("softplus", _i32), ("n", _i64), ("l", _i64), ("d", _i64), ("s", _i32),
                ("reserved", _i32), ("u_stride", _i64 * 2), ("delta_stride", _i64 * 2), ("b_stride", _i64 * 2),
                ("c_stride", _i64 * 2), ("gate_stride", _i64 * 2), ("dy_stride", _i64 * 2)]


class ScanInputs(ctypes.Structure):
    _fields_ = [(f, _vp) for f in ("u", "delta", "a", "b", "c", "skip", "gate", "delta_bias", "state", "lengths")]


class ScanGradPointers(ctypes.Structure):
    _fields_ = [(f, _vp) for f in ("u", "delta", "a", "b", "c", "skip", "gate", "delta_bias", "state")]


SEQ_EXPORTED = {
    "cnhwc_layer_norm_fwd": [_P(LayerNormDesc)] + [_vp] * 7,
    "cnhwc_layer_norm_bwd_workspace": [_P(LayerNormDesc), _i32, _P(_u64)],
    "cnhwc_layer_norm_bwd": [_P(LayerNormDesc)] + [_vp] * 9 + [_u64, _vp],
    "cnhwc_causal_conv_fwd": [_P(CausalConvDesc)] + [_vp] * 8,
    "cnhwc_causal_conv_bwd_workspace": [_P(CausalConvDesc), _P(_u64)],
    "cnhwc_causal_conv_bwd": [_P(CausalConvDesc)] + [_vp] * 12 + [_u64, _vp],
    "cnhwc_causal_conv_step": [_P(CausalConvDesc)] + [_vp] * 7,
    "cnhwc_scan_fwd_workspace": [_P(ScanDesc), _P(_u64)],
    "cnhwc_scan_fwd": [_P(ScanDesc), _P(ScanInputs), _vp, _vp, _vp, _u64, _vp],
    "cnhwc_scan_bwd_workspace": [_P(ScanDesc), _P(_u64)],
    "cnhwc_scan_bwd": [_P(ScanDesc), _P(ScanInputs), _vp, _vp, _P(ScanGradPointers), _vp, _u64, _vp],
    "cnhwc_scan_step": [_P(ScanDesc), _P(ScanInputs), _vp, _vp, _vp],
}
for _name, _args in SEQ_EXPORTED.items():
    _fn = getattr(lib, _name)
    _fn.restype, _fn.argtypes = ctypes.c_int, _args

ConvGrads = collections.namedtuple("ConvGrads", "x w bias state")
ScanGrads = collections.namedtuple("ScanGrads", "u delta a b c skip gate delta_bias state")


# ------------------------------------------------------------------ descriptors

def _norm_desc(dtype, w_dtype, n, l, c, xs, gs, eps):
    d = LayerNormDesc(dtype=dtype, w_dtype=w_dtype, n=n, l=l, c=c, eps=eps)
    d.x_stride[:], d.dy_stride[:] = xs, gs
    return d


def _conv_desc(dtype, act, n, l, c, k, xs, gs):
    d = CausalConvDesc(dtype=dtype, activation=act, n=n, l=l, c=c, k=k)
    d.x_stride[:], d.dy_stride[:] = xs, gs
    return d


def _scan_desc(dtype, softplus, n, l, d, s, us, ds, bs, cs, gs, ys):
    r = ScanDesc(dtype=dtype, softplus=softplus, n=n, l=l, d=d, s=s)
    r.u_stride[:], r.delta_stride[:], r.b_stride[:], r.c_stride[:] = us, ds, bs, cs
    r.gate_stride[:], r.dy_stride[:] = gs, ys
    return r


def _bytes(name, desc, *args):
    """Workspace bytes that the library asks for."""
    need = _u64()
    st = getattr(lib, name)(desc, *args, ctypes.byref(need))
    if st != 0:
        raise CnhwcError(st, name)
    return int(need.value)


def _activation(activation):
    if activation not in ACTIVATIONS:
        raise ValueError(f"activation must be one of {list(ACTIVATIONS)}")
    return ACTIVATIONS[activation]


# ------------------------------------------------------------------ layer norm

def layer_norm(x, weight=None, bias=None, eps=1e-5, *, return_stats=False, out=None):
    """y[..., C] = (x - mean) * rstd * weight + bias over the channels of each row,
    rstd = 1 / sqrt(var + eps).  weight and bias [C] have x's dtype or float32;
    with return_stats: (y, mean, rstd), the float32 statistics [...] that
    layer_norm_backward takes."""
    return _seq.layer_norm(x, weight, bias, eps, return_stats, out)


def layer_norm_backward(dy, x, mean, rstd, weight=None, *, workspace=None):
    """(dx, dweight, dbias) of layer_norm from dy and the statistics of the forward
    pass; dweight and dbias [C] have weight's dtype (both None without weight)."""
    return _seq.layer_norm_backward(dy, x, mean, rstd, weight, workspace)


def layer_norm_backward_workspace_bytes(x, weight=None):
    """Bytes of the workspace that layer_norm_backward needs for x [..., C] and weight."""
    if x.numel() == 0:
        return 0
    c, code = x.shape[-1], _DTYPE_CODE[x.dtype]
    desc = _norm_desc(code, code if weight is None else _DTYPE_CODE[weight.dtype], 1, x.numel() // c, c, (0, c), (0, c),
                      0.0)
    return _bytes("cnhwc_layer_norm_bwd_workspace", desc, int(weight is not None))


# ------------------------------------------------------------------ causal convolution

def causal_conv1d(x, w, bias=None, *, activation=None, state=None, lengths=None, return_state=False, out=None):
    """Depthwise causal conv1d: y[n,t,c] = act(bias[c] + sum_k w[c,k] X[n,t+k,c]), X
    being K-1 rows of state [N,K-1,C] (zeros if None) followed by x [N,L,C];
    w [C,K], K <= 8; activation None or "silu".  With return_state:
    (y, the state after the last valid position)."""
    return _seq.causal_conv1d(x, w, bias, _activation(activation), state, lengths, return_state, out)


def causal_conv1d_backward(dy, x, w, bias=None, *, activation=None, state=None, lengths=None, dstate=None,
                           workspace=None):
    """ConvGrads(x, w, bias, state) of causal_conv1d from dy [N,L,C] and, if given,
    dstate [N,K-1,C], the gradient of the returned state; bias and state are
    None where the forward pass had none."""
    return ConvGrads(*_seq.causal_conv1d_backward(dy, x, w, bias, _activation(activation), state, lengths, dstate,
                                                   workspace))


def causal_conv1d_backward_workspace_bytes(x, w):
    """Bytes of the workspace that causal_conv1d_backward needs for x [N,L,C] and w [C,K]."""
    if x.numel() == 0:
        return 0
    n, l, c = x.shape
    return _bytes("cnhwc_causal_conv_bwd_workspace",
                  _conv_desc(_DTYPE_CODE[x.dtype], 0, n, l, c, w.shape[1], (l * c, c), (l * c, c)))


def causal_conv1d_step(x, state, w, bias=None, *, activation=None, state_out=None, out=None):
    """causal_conv1d of one new token per sequence: x [N,C], y [N,C].  The state
    [N,K-1,C] moves on by the token, in place or into state_out."""
    return _seq.causal_conv1d_step(x, state, w, bias, _activation(activation), state_out, out)


# ------------------------------------------------------------------ selective scan

def selective_scan(u, delta, a, b, c, *, skip=None, gate=None, delta_bias=None, softplus=False, state=None,
                   lengths=None, return_state=False, out=None, workspace=None):
    """The selective state space scan: with D = softplus(delta + delta_bias) (the sum
    alone without softplus),

        h[n,t,d,s] = exp(D[n,t,d] a[d,s]) h[n,t-1,d,s] + D[n,t,d] u[n,t,d] b[n,t,s]
        y[n,t,d] = (sum_s c[n,t,s] h[n,t,d,s] + skip[d] u[n,t,d]) * silu(gate[n,t,d])

    u, delta, gate, y [N,L,D] and b, c [N,L,S] in one dtype; a [D,S], skip,
    delta_bias [D] and the states [N,D,S] in float32; S <= 64.  Absent skip,
    delta_bias and state count as 0, an absent gate leaves its factor out.  States
    that grow (D a > 0) by e^88 within a chunk of positions do not fit float32.
    With return_state: (y, the state after the last valid position)."""
    return _seq.selective_scan(u, delta, a, b, c, skip, gate, delta_bias, softplus, state, lengths, return_state, out,
                               workspace)


def selective_scan_backward(dy, u, delta, a, b, c, *, skip=None, gate=None, delta_bias=None, softplus=False,
                            state=None, lengths=None, dstate=None, workspace=None):
    """ScanGrads(u, delta, a, b, c, skip, gate, delta_bias, state) of selective_scan
    from dy [N,L,D] and, if given, dstate [N,D,S], the gradient of the returned
    state.  Those of inputs that were absent are None.  Nothing needs to be kept
    from the forward pass but its inputs."""
    return ScanGrads(*_seq.selective_scan_backward(dy, u, delta, a, b, c, skip, gate, delta_bias, softplus, state,
                                                    lengths, dstate, workspace))


def selective_scan_workspace_bytes(u, a, backward=False):
    """Bytes of the workspace that selective_scan (or its backward) needs for u [N,L,D] and a [D,S]."""
    if u.numel() == 0:
        return 0
    n, l, d = u.shape
    s = a.shape[1]
    wide, narrow = (l * d, d), (l * s, s)
    return _bytes("cnhwc_scan_bwd_workspace" if backward else "cnhwc_scan_fwd_workspace",
                  _scan_desc(_DTYPE_CODE[u.dtype], 0, n, l, d, s, wide, wide, narrow, narrow, wide, wide))


def selective_scan_step(u, delta, a, b, c, state, *, skip=None, gate=None, delta_bias=None, softplus=False,
                        state_out=None, out=None):
    """selective_scan of one new token per sequence: u, delta, gate, y [N,D], b, c
    [N,S].  The state [N,D,S] moves on by the token, in place or into state_out."""
    return _seq.selective_scan_step(u, delta, a, b, c, state, skip, gate, delta_bias, softplus, state_out, out)
