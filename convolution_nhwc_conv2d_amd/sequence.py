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
"""
import collections
import ctypes
import functools
import struct

import torch

from . import _DTYPE_CODE, CnhwcError, lib

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
    "cnhwc_scan_fwd": [_P(ScanDesc), _vp, _vp, _vp, _vp, _u64, _vp],
    "cnhwc_scan_bwd_workspace": [_P(ScanDesc), _P(_u64)],
    "cnhwc_scan_bwd": [_P(ScanDesc), _vp, _vp, _vp, _vp, _vp, _u64, _vp],
    "cnhwc_scan_step": [_P(ScanDesc), _vp, _vp, _vp, _vp],
}
for _name, _args in SEQ_EXPORTED.items():
    _fn = getattr(lib, _name)
    _fn.restype, _fn.argtypes = ctypes.c_int, _args

ConvGrads = collections.namedtuple("ConvGrads", "x w bias state")
ScanGrads = collections.namedtuple("ScanGrads", "u delta a b c skip gate delta_bias state")


# ------------------------------------------------------------------ helpers
#
# A single token's call takes a few microseconds on the GPU, so what is done per
# call here is kept short: descriptors are made once for a shape, and an
# argument is looked at in detail only when the quick test of it fails.

# The current stream and device as plain integers.
_stream = torch._C._cuda_getCurrentRawStream
_device = torch._C._cuda_getDevice


def _dtype(x, name="x"):
    """The dtype code of x, and x's device index."""
    if not isinstance(x, torch.Tensor) or not x.is_cuda:
        raise TypeError(f"{name} must be a GPU torch tensor")
    code = _DTYPE_CODE.get(x.dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {x.dtype}")
    return code, x.get_device()


def _like(t, name, dev, dtype, shape, dense=True):
    """Checks t against a device, a dtype and a shape; dense, or with a channel stride of 1."""
    try:
        if t.dtype is dtype and t.shape == shape and t.get_device() == dev:
            if t.is_contiguous() or (not dense and t.stride(-1) == 1):
                return t
    except AttributeError:
        pass
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.get_device() != dev:
        raise TypeError(f"{name} must be a torch tensor on cuda:{dev}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if dense:
        raise ValueError(f"{name} must be contiguous")
    if t.shape[-1] != 1:
        raise ValueError(f"{name} must have a channel stride of 1")
    return t


def _new(out, name, x, dev):
    """An output like x: the caller's, or a new dense one."""
    if out is None:
        return torch.empty_like(x) if x.is_contiguous() else torch.empty(x.shape, dtype=x.dtype, device=x.device)
    return _like(out, name, dev, x.dtype, x.shape)


def _ptr(t):
    return None if t is None else t.data_ptr()


_pack10, _pack9 = struct.Struct("10P").pack, struct.Struct("9P").pack  # ScanInputs, ScanGradPointers


def _adr(t):
    return 0 if t is None else t.data_ptr()


def _call(fn, dev, *args):
    """fn(*args, stream) on the device dev and its current stream."""
    if dev != _device():
        with torch.cuda.device(dev):
            st = fn(*args, _stream(dev))
    else:
        st = fn(*args, _stream(dev))
    if st != 0:
        raise CnhwcError(st, fn.__name__)


@functools.lru_cache(maxsize=4096)
def _bytes(name, desc_key, *args):
    """Workspace bytes that the library asks for (desc_key rebuilds the descriptor)."""
    make, key = desc_key
    need = _u64()
    st = getattr(lib, name)(make(*key), *args, ctypes.byref(need))
    if st != 0:
        raise CnhwcError(st, name)
    return int(need.value)


def _workspace(workspace, need, x, dev):
    if workspace is None:
        return torch.empty(need, dtype=torch.uint8, device=x.device) if need else None
    if not isinstance(workspace, torch.Tensor) or not workspace.is_cuda or workspace.get_device() != dev:
        raise TypeError(f"workspace must be a torch tensor on cuda:{dev}")
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return workspace


def _ws_args(ws):
    return (None, 0) if ws is None else (ws.data_ptr(), ws.numel() * ws.element_size())


def _rows(x, name):
    """x [..., C] as (n, l, c) and the strides of n and l, without a copy."""
    if x.dim() < 1:
        raise ValueError(f"{name} must be [..., C]")
    if x.stride(-1) != 1 and x.shape[-1] != 1:
        raise ValueError(f"{name} must have a channel stride of 1")
    if x.dim() == 3:
        return tuple(x.shape), (x.stride(0), x.stride(1))
    if x.dim() == 2:
        return (1, x.shape[0], x.shape[1]), (0, x.stride(0))
    if x.dim() == 1:
        return (1, 1, x.shape[0]), (0, 0)
    try:
        x = x.view(-1, x.shape[-2], x.shape[-1])
    except RuntimeError:
        raise ValueError(f"{name}: the leading dimensions must collapse to one stride") from None
    return tuple(x.shape), (x.stride(0), x.stride(1))


# ------------------------------------------------------------------ layer norm

@functools.lru_cache(maxsize=4096)
def _norm_desc(dtype, w_dtype, n, l, c, xs, gs, eps):
    d = LayerNormDesc(dtype=dtype, w_dtype=w_dtype, n=n, l=l, c=c, eps=eps)
    d.x_stride[:], d.dy_stride[:] = xs, gs
    return d


def _norm_params(weight, bias, x, dev):
    """The parameters' dtype: x's or float32."""
    if weight is None:
        if bias is not None:
            raise ValueError("bias needs weight")
        return x.dtype
    wd = weight.dtype if isinstance(weight, torch.Tensor) else None
    if wd is not x.dtype and wd is not torch.float32:
        raise TypeError(f"weight must be a {x.dtype} or float32 tensor")
    _like(weight, "weight", dev, wd, x.shape[-1:])
    if bias is not None:
        _like(bias, "bias", dev, wd, x.shape[-1:])
    return wd


def layer_norm(x, weight=None, bias=None, eps=1e-5, *, return_stats=False, out=None):
    """y[..., C] = (x - mean) * rstd * weight + bias over the channels of each row,
    rstd = 1 / sqrt(var + eps).  weight and bias [C] have x's dtype or float32;
    with return_stats: (y, mean, rstd), the float32 statistics [...] that
    layer_norm_backward takes."""
    code, dev = _dtype(x)
    (n, l, c), xs = _rows(x, "x")
    wd = _norm_params(weight, bias, x, dev)
    y = _new(out, "out", x, dev)
    mean = rstd = None
    if return_stats:
        mean = torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device)
        rstd = torch.empty_like(mean)
    if n * l > 0:
        _call(lib.cnhwc_layer_norm_fwd, dev, _norm_desc(code, _DTYPE_CODE[wd], n, l, c, xs, (0, 0), float(eps)),
              x.data_ptr(), _ptr(weight), _ptr(bias), y.data_ptr(), _ptr(mean), _ptr(rstd))
    return (y, mean, rstd) if return_stats else y


def layer_norm_backward(dy, x, mean, rstd, weight=None, *, workspace=None):
    """(dx, dweight, dbias) of layer_norm from dy and the statistics of the forward
    pass; dweight and dbias [C] have weight's dtype (both None without weight)."""
    code, dev = _dtype(x)
    (n, l, c), xs = _rows(x, "x")
    gs = _rows(_like(dy, "dy", dev, x.dtype, x.shape, dense=False), "dy")[1]
    _like(mean, "mean", dev, torch.float32, x.shape[:-1])
    _like(rstd, "rstd", dev, torch.float32, x.shape[:-1])
    wd = _norm_params(weight, None, x, dev)
    dx = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    dw = db = None
    if weight is not None:
        dw, db = torch.empty_like(weight), torch.empty_like(weight)
    if n * l == 0:
        return (dx, None, None) if dw is None else (dx, dw.zero_(), db.zero_())
    key = (code, _DTYPE_CODE[wd], n, l, c, xs, gs, 0.0)
    need = _bytes("cnhwc_layer_norm_bwd_workspace", (_norm_desc, key), int(dw is not None))
    ws = _workspace(workspace, need, x, dev)
    _call(lib.cnhwc_layer_norm_bwd, dev, _norm_desc(*key), dy.data_ptr(), x.data_ptr(), mean.data_ptr(),
          rstd.data_ptr(), _ptr(weight), dx.data_ptr(), _ptr(dw), _ptr(db), *_ws_args(ws))
    return dx, dw, db


def layer_norm_backward_workspace_bytes(x, weight=None):
    """Bytes of the workspace that layer_norm_backward needs for x and weight."""
    code, dev = _dtype(x)
    (n, l, c), xs = _rows(x, "x")
    if n * l == 0:
        return 0
    key = (code, _DTYPE_CODE[_norm_params(weight, None, x, dev)], n, l, c, xs, xs, 0.0)
    return _bytes("cnhwc_layer_norm_bwd_workspace", (_norm_desc, key), int(weight is not None))


# ------------------------------------------------------------------ causal convolution

@functools.lru_cache(maxsize=4096)
def _conv_desc(dtype, act, n, l, c, k, xs, gs):
    d = CausalConvDesc(dtype=dtype, activation=act, n=n, l=l, c=c, k=k)
    d.x_stride[:], d.dy_stride[:] = xs, gs
    return d


def _conv_check(x, w, bias, activation, state, lengths, dims):
    """Checks every input; (dtype code, device, activation code, K)."""
    code, dev = _dtype(x)
    if x.dim() != dims:
        raise ValueError("x must be [N,L,C]" if dims == 3 else "x must be [N,C]")
    c = x.shape[-1]
    if x.stride(-1) != 1 and c != 1:
        raise ValueError("x must have a channel stride of 1")
    if not isinstance(w, torch.Tensor) or w.dim() != 2 or w.shape[0] != c or w.shape[1] < 1:
        raise ValueError("w must be [C,K] with x's channels and K >= 1")
    act = ACTIVATIONS.get(activation)
    if act is None:
        raise ValueError(f"activation must be one of {list(ACTIVATIONS)}")
    dt, k = x.dtype, w.shape[1]
    _like(w, "w", dev, dt, w.shape)
    if bias is not None:
        _like(bias, "bias", dev, dt, (c,))
    if state is not None:
        _like(state, "state", dev, dt, (x.shape[0], k - 1, c))
    if lengths is not None:
        _like(lengths, "lengths", dev, torch.int32, x.shape[:1])
    return code, dev, act, k


def causal_conv1d(x, w, bias=None, *, activation=None, state=None, lengths=None, return_state=False, out=None):
    """Depthwise causal conv1d: y[n,t,c] = act(bias[c] + sum_k w[c,k] X[n,t+k,c]), X
    being K-1 rows of state [N,K-1,C] (zeros if None) followed by x [N,L,C];
    w [C,K], K <= 8; activation None or "silu".  With return_state:
    (y, the state after the last valid position)."""
    code, dev, act, k = _conv_check(x, w, bias, activation, state, lengths, 3)
    n, l, c = x.shape
    y = _new(out, "out", x, dev)
    last = torch.empty((n, k - 1, c), dtype=x.dtype, device=x.device) if return_state else None
    if n * l * c > 0:
        _call(lib.cnhwc_causal_conv_fwd, dev, _conv_desc(code, act, n, l, c, k, x.stride()[:2], (0, 0)), x.data_ptr(),
              w.data_ptr(), _ptr(bias), _ptr(state), _ptr(lengths), y.data_ptr(), _ptr(last))
    elif last is not None:
        last.zero_() if state is None else last.copy_(state)
    return (y, last) if return_state else y


def causal_conv1d_backward(dy, x, w, bias=None, *, activation=None, state=None, lengths=None, dstate=None,
                           workspace=None):
    """ConvGrads(x, w, bias, state) of causal_conv1d from dy [N,L,C] and, if given,
    dstate [N,K-1,C], the gradient of the returned state; bias and state are
    None where the forward pass had none."""
    code, dev, act, k = _conv_check(x, w, bias, activation, state, lengths, 3)
    n, l, c = x.shape
    _like(dy, "dy", dev, x.dtype, x.shape, dense=False)
    if dstate is not None:
        _like(dstate, "dstate", dev, x.dtype, (n, k - 1, c))
    dx, dw = torch.empty(x.shape, dtype=x.dtype, device=x.device), torch.empty_like(w)
    db = None if bias is None else torch.empty_like(bias)
    ds = None if state is None else torch.empty_like(state)
    if n * l * c == 0:
        if ds is not None:
            ds.zero_() if dstate is None else ds.copy_(dstate)
        return ConvGrads(dx, dw.zero_(), None if db is None else db.zero_(), ds)
    key = (code, act, n, l, c, k, x.stride()[:2], dy.stride()[:2])
    ws = _workspace(workspace, _bytes("cnhwc_causal_conv_bwd_workspace", (_conv_desc, key)), x, dev)
    _call(lib.cnhwc_causal_conv_bwd, dev, _conv_desc(*key), dy.data_ptr(), _ptr(dstate), x.data_ptr(), w.data_ptr(),
          _ptr(bias), _ptr(state), _ptr(lengths), dx.data_ptr(), dw.data_ptr(), _ptr(db), _ptr(ds), *_ws_args(ws))
    return ConvGrads(dx, dw, db, ds)


def causal_conv1d_backward_workspace_bytes(x, w):
    """Bytes of the workspace that causal_conv1d_backward needs for x and w."""
    code, _, _, k = _conv_check(x, w, None, None, None, None, 3)
    if x.numel() == 0:
        return 0
    key = (code, 0, *x.shape, k, x.stride()[:2], x.stride()[:2])
    return _bytes("cnhwc_causal_conv_bwd_workspace", (_conv_desc, key))


def causal_conv1d_step(x, state, w, bias=None, *, activation=None, state_out=None, out=None):
    """causal_conv1d of one new token per sequence: x [N,C], y [N,C].  The state
    [N,K-1,C] moves on by the token, in place or into state_out."""
    code, dev, act, k = _conv_check(x, w, bias, activation, state, None, 2)
    if state is None:
        raise ValueError("state is required")
    n, c = x.shape
    if state_out is None:
        state_out = state
    else:
        _like(state_out, "state_out", dev, x.dtype, state.shape)
    y = _new(out, "out", x, dev)
    if n * c > 0:
        _call(lib.cnhwc_causal_conv_step, dev, _conv_desc(code, act, n, 1, c, k, (x.stride(0), 0), (0, 0)),
              x.data_ptr(), state.data_ptr(), w.data_ptr(), _ptr(bias), y.data_ptr(), state_out.data_ptr())
    return y


# ------------------------------------------------------------------ selective scan

@functools.lru_cache(maxsize=4096)
def _scan_desc(dtype, softplus, n, l, d, s, us, ds, bs, cs, gs, ys):
    r = ScanDesc(dtype=dtype, softplus=softplus, n=n, l=l, d=d, s=s)
    r.u_stride[:], r.delta_stride[:], r.b_stride[:], r.c_stride[:] = us, ds, bs, cs
    r.gate_stride[:], r.dy_stride[:] = gs, ys
    return r


def _scan_check(u, delta, a, b, c, skip, gate, delta_bias, state, lengths, dims):
    """Checks every input; (dtype code, device, n, l, d, s)."""
    code, dev = _dtype(u, "u")
    if u.dim() != dims:
        raise ValueError("u must be [N,L,D]" if dims == 3 else "u must be [N,D]")
    shape, dt, f32 = u.shape, u.dtype, torch.float32
    n, d = shape[0], shape[-1]
    if not isinstance(a, torch.Tensor) or a.dim() != 2 or a.shape[0] != d or a.shape[1] < 1:
        raise ValueError("a must be [D,S] with u's channels and S >= 1")
    s = a.shape[1]
    of_states = shape[:-1] + (s,)
    _like(u, "u", dev, dt, shape, dense=False)
    _like(delta, "delta", dev, dt, shape, dense=False)
    _like(a, "a", dev, f32, a.shape)
    _like(b, "b", dev, dt, of_states, dense=False)
    _like(c, "c", dev, dt, of_states, dense=False)
    if skip is not None:
        _like(skip, "skip", dev, f32, (d,))
    if gate is not None:
        _like(gate, "gate", dev, dt, shape, dense=False)
    if delta_bias is not None:
        _like(delta_bias, "delta_bias", dev, f32, (d,))
    if state is not None:
        _like(state, "state", dev, f32, (n, d, s))
    if lengths is not None:
        _like(lengths, "lengths", dev, torch.int32, (n,))
    return code, dev, n, (shape[1] if dims == 3 else 1), d, s


def _scan_key(code, softplus, n, l, d, s, u, delta, b, c, gate, dy=None):
    """Arguments of _scan_desc; a stride of [N,C] or [N,L,C] tensors past their own is not looked at."""
    none = (0, 0)
    if u.dim() == 2:  # one token: the sequence strides alone
        return (code, 1 if softplus else 0, n, l, d, s, (u.stride(0), 0), (delta.stride(0), 0), (b.stride(0), 0),
                (c.stride(0), 0), none if gate is None else (gate.stride(0), 0), none)
    return (code, 1 if softplus else 0, n, l, d, s, u.stride()[:2], delta.stride()[:2], b.stride()[:2], c.stride()[:2],
            none if gate is None else gate.stride()[:2], none if dy is None else dy.stride()[:2])


def _scan_inputs(u, delta, a, b, c, skip, gate, delta_bias, state, lengths):
    return _pack10(u.data_ptr(), delta.data_ptr(), a.data_ptr(), b.data_ptr(), c.data_ptr(), _adr(skip), _adr(gate),
                   _adr(delta_bias), _adr(state), _adr(lengths))


def selective_scan(u, delta, a, b, c, *, skip=None, gate=None, delta_bias=None, softplus=False, state=None,
                   lengths=None, return_state=False, out=None, workspace=None):
    """The selective state space scan: with D = softplus(delta + delta_bias) (the sum
    alone without softplus),

        h[n,t,d,s] = exp(D[n,t,d] a[d,s]) h[n,t-1,d,s] + D[n,t,d] u[n,t,d] b[n,t,s]
        y[n,t,d] = (sum_s c[n,t,s] h[n,t,d,s] + skip[d] u[n,t,d]) * silu(gate[n,t,d])

    u, delta, gate, y [N,L,D] and b, c [N,L,S] in one dtype; a [D,S], skip,
    delta_bias [D] and the states [N,D,S] in float32; S <= 64.  Absent skip,
    delta_bias and state count as 0, an absent gate leaves its factor out.
    With return_state: (y, the state after the last valid position)."""
    code, dev, n, l, d, s = _scan_check(u, delta, a, b, c, skip, gate, delta_bias, state, lengths, 3)
    y = _new(out, "out", u, dev)
    last = torch.empty((n, d, s), dtype=torch.float32, device=u.device) if return_state else None
    if n * l * d > 0:
        key = _scan_key(code, softplus, n, l, d, s, u, delta, b, c, gate)
        ws = _workspace(workspace, _bytes("cnhwc_scan_fwd_workspace", (_scan_desc, key)), u, dev)
        ins = _scan_inputs(u, delta, a, b, c, skip, gate, delta_bias, state, lengths)
        _call(lib.cnhwc_scan_fwd, dev, _scan_desc(*key), ins, y.data_ptr(), _ptr(last), *_ws_args(ws))
    elif last is not None:
        last.zero_() if state is None else last.copy_(state)
    return (y, last) if return_state else y


def selective_scan_backward(dy, u, delta, a, b, c, *, skip=None, gate=None, delta_bias=None, softplus=False,
                            state=None, lengths=None, dstate=None, workspace=None):
    """ScanGrads(u, delta, a, b, c, skip, gate, delta_bias, state) of selective_scan
    from dy [N,L,D] and, if given, dstate [N,D,S], the gradient of the returned
    state.  Those of inputs that were absent are None.  Nothing needs to be kept
    from the forward pass but its inputs."""
    code, dev, n, l, d, s = _scan_check(u, delta, a, b, c, skip, gate, delta_bias, state, lengths, 3)
    _like(dy, "dy", dev, u.dtype, u.shape, dense=False)
    if dstate is not None:
        _like(dstate, "dstate", dev, torch.float32, (n, d, s))

    def like(t):
        return None if t is None else torch.empty(t.shape, dtype=t.dtype, device=t.device)
    r = ScanGrads(*(like(t) for t in (u, delta, a, b, c, skip, gate, delta_bias, state)))
    if n * l * d == 0:
        for t in r:
            if t is not None:
                t.zero_()
        if r.state is not None and dstate is not None:
            r.state.copy_(dstate)
        return r
    key = _scan_key(code, softplus, n, l, d, s, u, delta, b, c, gate, dy)
    ws = _workspace(workspace, _bytes("cnhwc_scan_bwd_workspace", (_scan_desc, key)), u, dev)
    ins = _scan_inputs(u, delta, a, b, c, skip, gate, delta_bias, state, lengths)
    _call(lib.cnhwc_scan_bwd, dev, _scan_desc(*key), ins, dy.data_ptr(), _ptr(dstate), _pack9(*map(_adr, r)),
          *_ws_args(ws))
    return r


def selective_scan_workspace_bytes(u, a, backward=False):
    """Bytes of the workspace that selective_scan (or its backward) needs for u and a."""
    if u.numel() == 0:
        return 0
    key = _scan_key(_dtype(u, "u")[0], False, *u.shape, a.shape[1], u, u, u, u, None, u)
    return _bytes("cnhwc_scan_bwd_workspace" if backward else "cnhwc_scan_fwd_workspace", (_scan_desc, key))


def selective_scan_step(u, delta, a, b, c, state, *, skip=None, gate=None, delta_bias=None, softplus=False,
                        state_out=None, out=None):
    """selective_scan of one new token per sequence: u, delta, gate, y [N,D], b, c
    [N,S].  The state [N,D,S] moves on by the token, in place or into state_out."""
    code, dev, n, _, d, s = _scan_check(u, delta, a, b, c, skip, gate, delta_bias, state, None, 2)
    if state is None:
        raise ValueError("state is required")
    if state_out is None:
        state_out = state
    else:
        _like(state_out, "state_out", dev, torch.float32, state.shape)
    y = _new(out, "out", u, dev)
    if n * d > 0:
        key = _scan_key(code, softplus, n, 1, d, s, u, delta, b, c, gate)
        ins = _scan_inputs(u, delta, a, b, c, skip, gate, delta_bias, state, None)
        _call(lib.cnhwc_scan_step, dev, _scan_desc(*key), ins, y.data_ptr(), state_out.data_ptr())
    return y
