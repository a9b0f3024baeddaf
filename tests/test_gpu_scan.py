"""The selective state space scan on the GPU against the 64-bit reference.

The bound's k: per position an exponential (its argument's rounding grows with
|D a|, at most about 4 here), a product and a sum, so 16 along each of L
positions; the gradient runs along them twice; softplus, gate and the sums over
states and channels add at most 128, the parameters' gradients every position.
"""
import numpy as np
import pytest
import torch

import seq_reference as R
from gpu_util import bits

pytestmark = pytest.mark.gpu

cn = pytest.importorskip("convolution_nhwc_conv2d_amd")

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SEQ = ("u", "delta", "b", "c", "gate")
NAMES = ("u", "delta", "a", "b", "c", "skip", "gate", "delta_bias", "state")


def _inputs(seed, n, l, d, s, dt, lengths=None, absent=()):
    g = np.random.default_rng(seed)
    t = DT[dt]
    r = lambda *sh, dtype=t, **kw: R.rand(g, *sh, **kw).to(dtype).cuda()
    f = torch.float32
    i = dict(u=r(n, l, d), delta=r(n, l, d, scale=0.7), a=-r(d, s, dtype=f).abs() - 0.05, b=r(n, l, s), c=r(n, l, s),
             skip=r(d, dtype=f), gate=r(n, l, d), delta_bias=r(d, dtype=f, scale=0.5, shift=-1.0),
             state=r(n, d, s, dtype=f), dy=r(n, l, d), dstate=r(n, d, s, dtype=f),
             lengths=None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda"))
    for name in absent:
        i[name] = None
    return i


def _kw(i, plus=True):
    return dict(skip=i["skip"], gate=i["gate"], delta_bias=i["delta_bias"], softplus=plus, state=i["state"],
                lengths=i["lengths"])


def _run(i, plus=True):
    return cn.selective_scan(i["u"], i["delta"], i["a"], i["b"], i["c"], return_state=True, **_kw(i, plus))


def _back(i, plus=True, **kw):
    return cn.selective_scan_backward(i["dy"], i["u"], i["delta"], i["a"], i["b"], i["c"], dstate=i["dstate"],
                                      **_kw(i, plus), **kw)


def _ref_args(i, plus):
    return [R.f64(i[k]) for k in ("u", "delta", "a", "b", "c", "skip", "gate", "delta_bias")] + [
        plus, R.f64(i["state"]), i["lengths"]]


def _forward(i, where, plus=True):
    y, last = _run(i, plus)
    ry, rl = R.scan(*_ref_args(i, plus))
    my, ml = R.scan(*_ref_args(i, plus), absolute=True)
    k = 16 * i["u"].shape[1] + 64
    R.check(y, ry, my, k, where + " y")
    R.check(last, rl, ml, k, where + " state")
    return y, last


def _backward(i, where, plus=True):
    r = _back(i, plus)
    args = [R.f64(i["dy"])] + _ref_args(i, plus) + [R.f64(i["dstate"])]
    want, mag = R.scan_backward(*args), R.scan_backward(*args, absolute=True)
    n, l = i["u"].shape[:2]
    k = 32 * l + 128
    for name in NAMES:
        got, key = getattr(r, name), "bias" if name == "delta_bias" else name
        if i[name] is None:
            assert got is None, name
            continue
        assert got.dtype == i[name].dtype
        R.check(got, want[key], mag[key], k + (n * l if name in ("a", "skip", "delta_bias") else 0), f"{where} d{name}")
    return r


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("s", [1, 3, 4, 5, 8, 13, 16, 24, 32, 48, 64])
def test_state_sizes(s, dt):
    for d in (70, 16):
        i = _inputs([1, s, d], 2, 27, d, s, dt)
        _forward(i, f"S {s} D {d}")
        _backward(i, f"S {s} D {d}")


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("l", [1, 2, 7, 8, 9, 16, 63, 64, 65, 200])
def test_lengths_of_sequences(l, dt):
    i = _inputs([2, l], 2, l, 33, 16, dt)
    _forward(i, f"L {l}")
    _backward(i, f"L {l}")


@pytest.mark.parametrize("d", [1, 2, 3, 4, 5, 63, 64, 65, 256, 257, 300])
def test_channel_counts(d):
    i = _inputs([3, d], 1, 20, d, 16, "bf16")
    _forward(i, f"D {d}")
    _backward(i, f"D {d}")


@pytest.mark.parametrize("plus", [True, False])
@pytest.mark.parametrize("absent", [("gate",), ("skip",), ("delta_bias",), ("state",), ("dstate",),
                                    ("gate", "skip", "delta_bias", "state", "dstate")])
def test_absent_inputs(absent, plus):
    i = _inputs([4], 2, 19, 40, 16, "f32", absent=absent)
    if not plus:  # D itself: small and positive, as a caller that has applied its own function gives it
        i["delta"] = i["delta"].abs() * 0.3
        if i["delta_bias"] is not None:
            i["delta_bias"] = i["delta_bias"].abs() * 0.3
    _forward(i, f"without {absent}", plus)
    _backward(i, f"without {absent}", plus)


@pytest.mark.parametrize("dt", ["f32", "f16"])
@pytest.mark.parametrize("state", [True, False])
def test_ragged(dt, state):
    """Lengths of none, one, inside and on chunk bounds, all, and beyond both ends;
    what stands past them (NaN, infinity) changes nothing."""
    lengths = [0, 1, 7, 64, 65, 150, 999, -3]
    i = _inputs([5], len(lengths), 150, 36, 16, dt, lengths=lengths, absent=() if state else ("state",))
    first = _forward(i, "ragged") + tuple(_backward(i, "ragged"))
    for n, m in enumerate(lengths):
        m = min(max(m, 0), 150)
        assert not first[0][n, m:].any()
        for name in SEQ:
            assert not first[2 + NAMES.index(name)][n, m:].any(), name
            i[name][n, m:] = float("nan") if name != "b" else float("inf")
        i["dy"][n, m:] = float("nan")
    again = _run(i) + tuple(_back(i))
    for p, q in zip(first, again):
        assert p is None and q is None or torch.equal(bits(p), bits(q))


@pytest.mark.parametrize("dt", list(DT))
def test_strided_and_unaligned(dt):
    """u and gate as halves of one projection, b and c inside another, every
    second position, odd offsets, b and c shared by the sequences."""
    g = np.random.default_rng(6)
    ug, bc = R.rand(g, 2, 44, 161).to(DT[dt]).cuda(), R.rand(g, 2, 44, 77).to(DT[dt]).cuda()
    cuts = {"halves": lambda t, o, c: t[:, :22, o:o + c], "positions": lambda t, o, c: t[:, ::2, o:o + c],
            "shared": lambda t, o, c: t[:1, :22, o:o + c].expand(2, 22, c)}
    for name, cut in cuts.items():
        i = _inputs([6], 2, 22, 80, 16, dt)
        i.update(u=cut(ug, 0, 80), gate=cut(ug, 81, 80), b=cut(bc, 20, 16), c=cut(bc, 37, 16), dy=cut(ug, 40, 80))
        _forward(i, name)
        _backward(i, name)
    i = _inputs([6], 2, 22, 80, 16, dt)
    shift = torch.zeros(80 * 16 + 1, device="cuda")  # a off its 16-byte alignment
    shift[1:] = i["a"].flatten()
    i["a"] = shift[1:].view(80, 16)
    _forward(i, "a unaligned")
    _backward(i, "a unaligned")


def test_offsets_past_32_bits():
    far = (1 << 31) + 64
    buf = torch.empty(far + 256, dtype=torch.bfloat16, device="cuda")
    i = _inputs([7], 1, 2, 64, 16, "bf16")
    x = buf.as_strided((1, 2, 64), (far, far, 1))
    x.copy_(i["u"])
    i.update({k: x for k in ("u", "delta", "gate", "dy")}, b=x[..., :16], c=x[..., 16:32])
    _forward(i, "far")
    _backward(i, "far")


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("s", [3, 8, 16, 40])
def test_tokens_and_parts_give_the_prompt(s, dt):
    """Token by token (in place and into another buffer): the same bits as the
    prompt in one chunk; a prompt in two parts: the reference again."""
    i = _inputs([8, s], 3, 12, 45, s, dt)
    y, last = _forward(i, "prompt")
    kw = dict(skip=i["skip"], delta_bias=i["delta_bias"], softplus=True)
    state, other = i["state"].clone(), torch.empty_like(i["state"])
    for t in range(12):
        args = [i[k][:, t] if k in SEQ else i[k] for k in ("u", "delta", "a", "b", "c")]
        before = state.clone()
        z = cn.selective_scan_step(*args, state, gate=i["gate"][:, t], state_out=other, **kw)
        assert torch.equal(bits(state), bits(before))
        z2 = cn.selective_scan_step(*args, state, gate=i["gate"][:, t], **kw)
        assert torch.equal(bits(z), bits(y[:, t])) and torch.equal(bits(z2), bits(z)) and torch.equal(bits(state), bits(other))
    assert torch.equal(bits(state), bits(last))
    parts = {k: (v[:, :5] if k in SEQ else v) for k, v in i.items()}
    y1, s1 = _run(parts)
    parts = {k: (v[:, 5:] if k in SEQ else v) for k, v in i.items()}
    y2, s2 = _run(dict(parts, state=s1))
    assert torch.equal(bits(torch.cat([y1, y2], 1)), bits(y)) and torch.equal(bits(s2), bits(last))


def test_extreme_steps():
    """Steps so long that the state is forgotten (D 60), and none at all: exact limits, nothing non-finite."""
    i = _inputs([9], 1, 30, 64, 16, "f32", absent=("gate", "delta_bias"))
    i["a"] = i["a"] - 2.0
    i["delta"][:, 10:20] = 60.0
    i["delta"][:, 20:] = -200.0
    y, last = _run(i)
    h = 60.0 * R.f64(i["u"])[0, 19][:, None] * R.f64(i["b"])[0, 19][None, :]  # all that is left of the state
    R.check(last[0], h, h.abs(), 64, "state")
    r = _back(i)
    for name, t in zip(NAMES, r):
        assert t is None or bool(torch.isfinite(t).all()), name
    assert not r.delta[:, 20:].any()  # softplus is flat there in 32 bits


@pytest.mark.parametrize("lengths", [None, [23, 9]])
def test_gradient_against_differences(lengths):
    """<gradient, v> against central differences of the 64-bit forward pass."""
    i = _inputs([10], 2, 23, 12, 16, "f32", lengths=lengths)
    r = _backward(i, "differences")
    ins = {k: R.f64(i[k]) for k in NAMES}
    f = lambda u, delta, a, b, c, skip, gate, delta_bias, state: R.scan(u, delta, a, b, c, skip, gate, delta_bias, True,
                                                                        state, lengths and torch.tensor(lengths))
    args = [R.f64(i["dy"])] + _ref_args(i, True) + [R.f64(i["dstate"])]
    mag = R.scan_backward(*args, absolute=True)
    for name in NAMES:
        num, v = R.directional(f, ins, name, (R.f64(i["dy"]), R.f64(i["dstate"])))
        got = R.f64(getattr(r, name))
        m = mag["bias" if name == "delta_bias" else name]
        bound = float(((R.EPS * got.abs() + (32 * 23 + 174) * R.EPS * m) * v.abs()).sum())
        assert abs(num - float((got * v).sum())) <= bound + 1e-6 * abs(num), name


def test_same_bits_on_every_call_and_nothing_past_the_outputs():
    i = _inputs([11], 2, 300, 130, 16, "bf16", lengths=[300, 77])
    y0, s0 = _run(i)
    first = _back(i)
    need_f = cn.selective_scan_workspace_bytes(i["u"], i["a"])
    need = cn.selective_scan_workspace_bytes(i["u"], i["a"], backward=True)
    buf = torch.full((max(need, need_f) + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    out = torch.full((y0.numel() + 2048,), float("nan"), dtype=y0.dtype, device="cuda")
    for _ in range(3):
        y, s = cn.selective_scan(i["u"], i["delta"], i["a"], i["b"], i["c"], return_state=True, workspace=buf[:need_f],
                                 out=out[:y0.numel()].view(y0.shape), **_kw(i))
        torch.cuda.synchronize()
        assert torch.equal(bits(y), bits(y0)) and torch.equal(bits(s), bits(s0))
        assert bool((buf[need_f:] == 0xA5).all()) and bool(torch.isnan(out[y0.numel():].float()).all())
        again = _back(i, workspace=buf[:need])
        torch.cuda.synchronize()
        assert all(torch.equal(bits(p), bits(q)) for p, q in zip(first, again))
        assert bool((buf[need:] == 0xA5).all())
        buf.fill_(0xA5)
    with pytest.raises(cn.CnhwcError) as e:
        _back(i, workspace=buf[:need - 1])
    assert e.value.name == "WORKSPACE_TOO_SMALL"


def test_two_streams_at_once():
    """Calls queued on two streams give the bits that each gives alone."""
    ins = [_inputs([12, j], 2, 150, 90, 16, "f16") for j in range(2)]
    alone = [_run(i) + tuple(_back(i)) for i in ins]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [None, None]
    for j in range(2):
        with torch.cuda.stream(streams[j]):
            got[j] = _run(ins[j]) + tuple(_back(ins[j]))
    torch.cuda.synchronize()
    for g, a in zip(got, alone):
        assert all(torch.equal(bits(p), bits(q)) for p, q in zip(g, a))


def test_graph_replays():
    """A token step of convolution and scan, and a backward pass, as a graph: every replay gives the eager bits."""
    i = _inputs([13], 2, 90, 64, 16, "bf16")
    g = np.random.default_rng(13)
    x, w = R.rand(g, 2, 64).bfloat16().cuda(), R.rand(g, 64, 4).bfloat16().cuda()
    conv_state, state = torch.zeros(2, 3, 64, dtype=torch.bfloat16, device="cuda"), i["state"].clone()
    tok = {k: i[k][:, 0].clone() for k in SEQ}

    def token(conv_state, state):
        u = cn.causal_conv1d_step(x, conv_state, w, activation="silu")
        return cn.selective_scan_step(u, tok["delta"], i["a"], tok["b"], tok["c"], state, skip=i["skip"],
                                      gate=tok["gate"], delta_bias=i["delta_bias"], softplus=True)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        token(conv_state.clone(), state.clone())
        want_grads = _back(i)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = token(conv_state, state)
        grads = _back(i)
    eager_conv, eager_state = torch.zeros_like(conv_state), i["state"].clone()
    conv_state.zero_()
    state.copy_(i["state"])
    for _ in range(4):
        want = token(eager_conv, eager_state)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(bits(y), bits(want)) and torch.equal(bits(state), bits(eager_state))
        assert torch.equal(bits(conv_state), bits(eager_conv))
        assert all(torch.equal(bits(p), bits(q)) for p, q in zip(grads, want_grads))


def test_empty_and_refusals():
    i = _inputs([14], 2, 5, 8, 16, "f32")
    none = {k: (v[:, :0] if k in SEQ + ("dy",) else v) for k, v in i.items()}
    y, last = _run(none)
    assert y.shape == (2, 0, 8) and torch.equal(last, i["state"])
    r = _back(none)
    assert torch.equal(r.state, i["dstate"]) and not r.a.any() and not r.skip.any()
    run = lambda **kw: _run(dict(i, **kw))
    wide = torch.zeros(8, 65, device="cuda")
    for bad, kind in ((lambda: run(u=i["u"][0]), ValueError), (lambda: run(u=i["u"].cpu()), TypeError),
                      (lambda: run(delta=i["delta"].half()), TypeError), (lambda: run(delta=i["delta"][:, :4]), ValueError),
                      (lambda: run(a=i["a"][:4]), ValueError), (lambda: run(a=i["a"].half()), TypeError),
                      (lambda: run(b=i["b"][..., :8]), ValueError), (lambda: run(c=i["c"].transpose(1, 2)), ValueError),
                      (lambda: run(skip=i["skip"][:3]), ValueError), (lambda: run(gate=i["gate"].bfloat16()), TypeError),
                      (lambda: run(state=i["state"].half()), TypeError), (lambda: run(state=i["state"][:1]), ValueError),
                      (lambda: run(lengths=torch.zeros(2, dtype=torch.int64, device="cuda")), TypeError),
                      (lambda: run(a=wide, b=torch.zeros(2, 5, 65, device="cuda"), c=torch.zeros(2, 5, 65, device="cuda"),
                                   state=torch.zeros(2, 8, 65, device="cuda")), cn.CnhwcError),
                      (lambda: cn.selective_scan(i["u"], i["delta"], i["a"], i["b"], i["c"], out=i["u"]), cn.CnhwcError),
                      (lambda: cn.selective_scan_step(i["u"][:, 0], i["delta"][:, 0], i["a"], i["b"][:, 0], i["c"][:, 0], None),
                       ValueError),
                      (lambda: cn.selective_scan_backward(i["dy"][:1], i["u"], i["delta"], i["a"], i["b"], i["c"]), ValueError)):
        with pytest.raises(kind):
            bad()
