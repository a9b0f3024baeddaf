"""The scan at sizes whose chunks, joins and token batches small ones do not
have, against the batched 64-bit reference on the GPU.

A sequence is cut by the wavefronts of the call: 64 channels to one (32 above 16
states, 16 above 32), four to a workgroup.  Forward: chunks of L times the
wavefronts of one position over 4096, at least 16 positions (32 from L = 1536),
one chunk from 1024 wavefronts on; 16 chunks are joined at a time.  Backward: over 2048,
16 to 128 positions.  Decays are slow, so states cross many chunks.  Bounds as for
the small sizes: 16 roundings a position forward, 32 backward.
"""
import pytest
import torch

import seq_reference as R
import seq_reference_batched as B
from gpu_util import bits

pytestmark = pytest.mark.gpu

cn = pytest.importorskip("convolution_nhwc_conv2d_amd")

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
NAMES = ("u", "delta", "a", "b", "c", "skip", "gate", "delta_bias", "state")


def _inputs(seed, n, l, d, s, dt, lengths=None):
    g = torch.Generator(device="cuda").manual_seed(seed)
    f = torch.float32
    r = lambda *sh, dtype=DT[dt], scale=1.0: (torch.randn(sh, generator=g, device="cuda") * scale).to(dtype)
    return dict(u=r(n, l, d), delta=r(n, l, d, scale=0.7), a=-r(d, s, dtype=f, scale=0.1).abs() - 0.005, b=r(n, l, s),
                c=r(n, l, s), skip=r(d, dtype=f), gate=r(n, l, d), delta_bias=r(d, dtype=f, scale=0.5) - 1.0,
                state=r(n, d, s, dtype=f), dy=r(n, l, d), dstate=r(n, d, s, dtype=f),
                lengths=None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda"))


def _args(i):
    w = lambda t: t.double()
    return [w(i[k]) for k in ("u", "delta", "a", "b", "c", "skip", "gate", "delta_bias")] + [True, w(i["state"]),
                                                                                             i["lengths"]]


def _kw(i):
    return dict(skip=i["skip"], gate=i["gate"], delta_bias=i["delta_bias"], softplus=True, state=i["state"],
                lengths=i["lengths"])


def _check(got, ref, mag, k, where):
    R.check(got, ref.cpu(), mag.cpu(), k, where)


FORWARD = [
    # chunks of 16, several workgroups along the channels, every lane shape
    ("f32", 2, 100, 300, 4, None), ("f16", 2, 100, 300, 8, [100, 41]), ("bf16", 2, 131, 300, 32, None),
    ("f32", 2, 100, 300, 64, [67, 100]), ("bf16", 1, 129, 520, 16, None),
    # 19 and 70 chunks: more than are joined at a time
    ("f32", 3, 300, 300, 16, [300, 17, 259]), ("bf16", 1, 2230, 300, 16, None), ("f16", 2, 300, 90, 64, [300, 273]),
    # chunks of 24, 32 and 40
    ("f32", 40, 300, 300, 16, None), ("f16", 8, 1600, 270, 16, [1600, 1599, 0, 1, 31, 32, 33, 1000]),
    ("bf16", 64, 300, 300, 8, None),
    # one chunk
    ("f32", 130, 90, 300, 16, None), ("bf16", 60, 70, 300, 64, None),
]


@pytest.mark.parametrize("dt,n,l,d,s,lengths", FORWARD, ids=lambda v: "ragged" if isinstance(v, list) else str(v))
def test_forward(dt, n, l, d, s, lengths):
    i = _inputs(1, n, l, d, s, dt, lengths)
    y, last = cn.selective_scan(i["u"], i["delta"], i["a"], i["b"], i["c"], return_state=True, **_kw(i))
    ry, rl = B.scan(*_args(i))
    my, ml = B.scan(*_args(i), absolute=True)
    _check(y, ry, my, 16 * l + 64, "y")
    _check(last, rl, ml, 16 * l + 64, "state")


BACKWARD = [
    # chunks of 24 and 40 in one workgroup's width; tiles from the third on have kept states
    ("bf16", 12, 1024, 70, 16, None), ("f32", 5, 4096, 64, 4, [4096, 1, 0, 2500, 4095]),
    # chunks of 32, 72 and 128, several workgroups along the channels
    ("f16", 6, 1030, 300, 16, [1030, 1, 0, 1029, 513, 64]), ("f32", 8, 1400, 300, 32, None),
    ("bf16", 16, 2100, 300, 16, [2100 - 131 * j for j in range(15)] + [0]), ("f16", 8, 2060, 200, 64, None),
    ("f32", 16, 2060, 272, 8, None),
    # chunks of 16, more than are joined at a time
    ("f32", 2, 700, 300, 16, [700, 283]),
]


@pytest.mark.parametrize("dt,n,l,d,s,lengths", BACKWARD, ids=lambda v: "ragged" if isinstance(v, list) else str(v))
def test_backward(dt, n, l, d, s, lengths):
    i = _inputs(2, n, l, d, s, dt, lengths)
    r = cn.selective_scan_backward(i["dy"], i["u"], i["delta"], i["a"], i["b"], i["c"], dstate=i["dstate"], **_kw(i))
    args = [i["dy"].double()] + _args(i) + [i["dstate"].double()]
    mag = {k: v.cpu() for k, v in B.scan_backward(*args, absolute=True).items()}
    want = B.scan_backward(*args)
    k = 32 * l + 128
    for name in NAMES:
        key = "bias" if name == "delta_bias" else name
        _check(getattr(r, name), want[key], mag[key], k + (n * l if name in ("a", "skip", "delta_bias") else 0), "d" + name)
    if lengths is not None:
        for j, m in enumerate(lengths):
            for name in ("u", "delta", "b", "c", "gate"):
                assert not getattr(r, name)[j, m:].any(), name


# two sequences to a thread: more than 2048 workgroups with one; odd counts end in half a pair
@pytest.mark.parametrize("dt,n,d,s", [("f16", 33, 4096, 16), ("f32", 35, 4100, 16), ("bf16", 17, 4096, 32), ("f32", 9, 4096, 64),
                                      ("bf16", 33, 4100, 13), ("f16", 11, 4099, 48), ("f16", 32, 4096, 16), ("bf16", 33, 4097, 3)])
def test_tokens(dt, n, d, s):
    i = _inputs(3, n, 2, d, s, dt)
    state, other = i["state"].clone(), torch.empty_like(i["state"])
    for t in range(2):
        tok = {k: i[k][:, t:t + 1] for k in ("u", "delta", "b", "c", "gate")}
        one = dict(i, **tok, state=state)
        ry, rl = B.scan(*_args(one))
        my, ml = B.scan(*_args(one), absolute=True)
        kw = dict(skip=i["skip"], gate=tok["gate"][:, 0], delta_bias=i["delta_bias"], softplus=True)
        call = lambda **to: cn.selective_scan_step(tok["u"][:, 0], tok["delta"][:, 0], i["a"], tok["b"][:, 0], tok["c"][:, 0],
                                                   state, **kw, **to)
        before = state.clone()
        y = call(state_out=other)
        assert torch.equal(bits(state), bits(before))
        y2 = call()
        assert torch.equal(bits(y2), bits(y)) and torch.equal(bits(state), bits(other))
        _check(y, ry[:, 0], my[:, 0], 80, f"token {t} y")
        _check(state, rl, ml, 80, f"token {t} state")
