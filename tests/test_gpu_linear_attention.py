"""Linear attention on the GPU against the 64-bit reference, element by element.

The bound's k, in units of 2^-24 of the magnitude of an output's terms:
  - float32: a position adds a product and a sum, its decay's power is off by a
    few units; sums over 256 channels, 64 positions of a chunk and over the chunks
    add one rounding each: 2 L + 512.
  - 16-bit outputs: an operand of a product (the products of q and k under their
    decays, the state that a chunk starts from) may be rounded to the type once
    before the second product: u of each term, 2^16 (bf16) or 2^13 (f16) units.
  - the states and the decay's gradient are float32 whatever the inputs are: 2 L + 512
    again, and the decay's gradient sums the positions and sequences in 32 bits.
"""
import numpy as np
import pytest
import torch

import attention_reference as A
import seq_reference as R
from gpu_util import bits

pytestmark = pytest.mark.gpu

cn = pytest.importorskip("convolution_nhwc_conv2d_amd")

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
OPERAND = {"f32": 0, "f16": 1 << 13, "bf16": 1 << 16}
NAMES = ("q", "k", "v", "log_decay", "state")


def _inputs(seed, n, l, h, dk, dv, dt, lengths=None, state=True, life=None):
    g = np.random.default_rng(seed)
    r = lambda *sh, dtype=DT[dt], **kw: R.rand(g, *sh, **kw).to(dtype).cuda()
    f = torch.float32
    decay = -torch.from_numpy(np.exp(g.uniform(np.log(2e-4), np.log(0.7), h)).astype(np.float32)).cuda()
    if life is not None:
        decay = torch.full((h,), -np.log(2.0) / life, device="cuda")
    return dict(q=r(n, l, h, dk), k=r(n, l, h, dk), v=r(n, l, h, dv), log_decay=decay, dy=r(n, l, h, dv),
                state=r(n, h, dk, dv, dtype=f) if state else None, dstate=r(n, h, dk, dv, dtype=f) if state else None,
                scale=dk ** -0.5, dt=dt,
                lengths=None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda"))


def _run(i, **kw):
    return cn.linear_attention(i["q"], i["k"], i["v"], i["log_decay"], scale=i["scale"], state=i["state"],
                               lengths=i["lengths"], return_state=True, **kw)


def _back(i, decay_grad=True, **kw):
    return cn.linear_attention_backward(i["dy"], i["q"], i["k"], i["v"], i["log_decay"], scale=i["scale"],
                                        state=i["state"], lengths=i["lengths"], dstate=i["dstate"],
                                        decay_grad=decay_grad, **kw)


def _args(i):
    return [A.wide(i[k]) for k in ("q", "k", "v", "log_decay")] + [i["scale"], A.wide(i["state"]), i["lengths"]]


def _abs(args):
    """Absolute values, but for the decays."""
    return args[:0] + [a.abs() if torch.is_tensor(a) and a.is_floating_point() and a.dim() != 1 else a for a in args]


def _check(got, ref, mag, k, where):
    R.check(got, ref.cpu(), mag.cpu(), k, where)


def _forward(i, where):
    y, last = _run(i)
    ry, rl = A.attention(*_args(i))
    my, ml = A.attention(*_abs(_args(i)))
    k = 2 * i["q"].shape[1] + 512
    _check(y, ry, my, k + OPERAND[i["dt"]], where + " y")
    _check(last, rl, ml, k, where + " state")
    return y, last


def _backward(i, where, **kw):
    r = _back(i, **kw)
    args = [A.wide(i["dy"])] + _args(i)
    want = A.attention_backward(*args, A.wide(i["dstate"]))
    mag = A.attention_backward(*_abs(args), None if i["dstate"] is None else A.wide(i["dstate"]).abs())
    n, l = i["q"].shape[:2]
    k = 2 * l + 512
    for name in ("q", "k", "v"):
        _check(getattr(r, name), want[name], mag[name], k + OPERAND[i["dt"]], f"{where} d{name}")
    _check(r.log_decay, want["log_decay"], mag["log_decay"], k + n * l, where + " dlog_decay")
    if i["state"] is None:
        assert r.state is None
    else:
        _check(r.state, want["state"], mag["state"], k, where + " dstate")
    return r


DIMS = [(1, 1), (3, 5), (16, 16), (17, 33), (32, 64), (48, 100), (64, 32), (64, 64), (64, 96), (80, 72), (100, 128),
        (128, 64), (128, 128), (128, 200), (192, 40), (256, 256), (250, 130)]


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("dk,dv", DIMS)
def test_dimensions(dk, dv, dt):
    i = _inputs([1, dk, dv], 2, 70, 2, dk, dv, dt)
    _forward(i, f"{dk}x{dv}")
    _backward(i, f"{dk}x{dv}")


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("l", [1, 2, 3, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 200, 257, 520])
def test_lengths_of_sequences(l, dt):
    i = _inputs([2, l], 2, l, 3, 64, 48, dt, state=l % 2 == 1)
    _forward(i, f"L {l}")
    _backward(i, f"L {l}")


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("n,l,h", [(1, 4096, 1), (1, 3001, 2), (3, 1500, 5), (9, 700, 8)])
def test_long_and_many(n, l, h, dt):
    """Sequences in several parts, a half-life of 4096 positions among the decays."""
    i = _inputs([3, n, l], n, l, h, 64, 64, dt, state=n == 1)
    i["log_decay"][0] = -np.log(2.0) / 4096
    _forward(i, f"{n}x{l}x{h}")
    _backward(i, f"{n}x{l}x{h}")


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("state", [True, False])
def test_ragged(dt, state):
    """Lengths of none, one, inside and on tile bounds, all, and beyond both ends; what
    stands past them (NaN, infinity) changes nothing."""
    lengths = [0, 1, 15, 64, 65, 150, 999, -3]
    i = _inputs([4], len(lengths), 150, 3, 40, 56, dt, lengths=lengths, state=state)
    first = _forward(i, "ragged") + tuple(_backward(i, "ragged"))
    for n, m in enumerate(lengths):
        m = min(max(m, 0), 150)
        for t in (first[0], *first[2:5]):
            assert not t[n, m:].any()
        if state and m == 0:
            assert torch.equal(first[1][n], i["state"][n]) and torch.equal(first[6][n], i["dstate"][n])
        for name in ("q", "k", "v", "dy"):
            i[name][n, m:] = float("nan") if name != "k" else float("inf")
    again = _run(i) + tuple(_back(i))
    for p, q in zip(first, again):
        assert p is None and q is None or torch.equal(bits(p), bits(q))


@pytest.mark.parametrize("dt", list(DT))
def test_strided_and_shared(dt):
    """q, k and v inside one projection's rows, odd offsets, every second position,
    transposed heads, and keys that all heads share."""
    g = np.random.default_rng(5)
    rows = R.rand(g, 2, 44, 700).to(DT[dt]).cuda()
    cuts = {"rows": lambda o, d: rows[:, :22, o:o + 3 * d].unflatten(-1, (3, d)),
            "odd": lambda o, d: rows[:, :22, o + 1:o + 1 + 3 * d].unflatten(-1, (3, d)),
            "positions": lambda o, d: rows[:, ::2, o:o + 3 * d].unflatten(-1, (3, d)),
            "transposed": lambda o, d: rows[:, :, :3 * d].reshape(2, 3, 44, d)[:, :, :22].transpose(1, 2)}
    for name, cut in cuts.items():
        i = _inputs([5], 2, 22, 3, 64, 48, dt)
        i.update(q=cut(0, 64), k=cut(192, 64), v=cut(384, 48), dy=cut(528, 48))
        _forward(i, name)
        _backward(i, name)
    i = _inputs([5], 2, 22, 3, 64, 48, dt)
    i.update(k=rows[:, :22, :64].unflatten(-1, (1, 64)).expand(2, 22, 3, 64),
             q=rows[:1, :22, :192].unflatten(-1, (3, 64)).expand(2, 22, 3, 64),
             dy=rows[:, :1, :1].unsqueeze(-1).expand(2, 22, 3, 1)[..., :1].contiguous().expand(2, 22, 3, 1).repeat(1, 1, 1, 48))
    _forward(i, "shared")
    _backward(i, "shared")


def test_offsets_past_32_bits():
    far = (1 << 31) + 64
    buf = torch.empty(far + 256, dtype=torch.bfloat16, device="cuda")
    i = _inputs([6], 1, 2, 1, 64, 64, "bf16")
    x = buf.as_strided((1, 2, 1, 64), (far, far, 64, 1))
    x.copy_(i["q"])
    i.update({k: x for k in ("q", "k", "v", "dy")})
    _forward(i, "far")
    _backward(i, "far")


@pytest.mark.parametrize("dt", list(DT))
def test_decays_at_their_ends(dt):
    """None (0), at once (minus infinity), so fast that nothing is left of the last but one
    position, slower than 32 bits tell from none, and a little growth."""
    i = _inputs([7], 2, 140, 6, 32, 48, dt)
    i["log_decay"] = torch.tensor([0.0, float("-inf"), -200.0, -1e-9, -20.0, 1e-3], device="cuda")
    j = dict(i, log_decay=i["log_decay"].clamp(min=-1e4))  # the reference's exp(g) is 0 there too
    y, last = _run(i)
    ry, rl = A.attention(*_args(j))
    my, ml = A.attention(*_abs(_args(j)))
    k = 2 * 140 + 512
    _check(y, ry, my, k + OPERAND[dt], "y")
    _check(last, rl, ml, k, "state")
    r = _back(i)
    want = A.attention_backward(A.wide(i["dy"]), *_args(j), A.wide(i["dstate"]))
    mag = A.attention_backward(*_abs([A.wide(i["dy"])] + _args(j)), A.wide(i["dstate"]).abs())
    for name in NAMES:
        more = OPERAND[dt] if name in ("q", "k", "v") else 2 * 140
        _check(getattr(r, name), want[name], mag[name], k + more, "d" + name)


def test_slow_decay_over_many_tokens():
    """4000 tokens at a half-life of 4000: the power of the decay keeps its digits."""
    n = 4000
    state = torch.ones(1, 1, 2, 2, device="cuda")
    z = torch.zeros(1, 1, 2, device="cuda")
    g = torch.tensor([-np.log(2.0) / n], dtype=torch.float32, device="cuda")
    for _ in range(n):
        cn.linear_attention_step(z, z, z, g, state)
    want = float(torch.exp(g.double() * n))
    assert (state.double() / want - 1).abs().max() < n * 2.0 ** -25 + 2.0 ** -22


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("dk,dv", [(1, 1), (3, 5), (33, 40), (64, 64), (64, 100), (128, 128), (200, 72), (256, 256)])
def test_tokens_follow_the_prompt(dk, dv, dt):
    """A prompt, then tokens (in place and into another buffer): the reference again."""
    i = _inputs([8, dk, dv], 3, 20, 2, dk, dv, dt)
    ry, rl = A.attention(*_args(i))
    my, ml = A.attention(*_abs(_args(i)))
    part = {k: (v[:, :12] if k in ("q", "k", "v") else v) for k, v in i.items()}
    _, state = _run(part)
    other = torch.empty_like(state)
    k = 2 * 20 + 512
    for t in range(12, 20):
        a = [i[x][:, t] for x in ("q", "k", "v")]
        before = state.clone()
        y = cn.linear_attention_step(*a, i["log_decay"], state, scale=i["scale"], state_out=other)
        assert torch.equal(bits(state), bits(before))
        y2 = cn.linear_attention_step(*a, i["log_decay"], state, scale=i["scale"])
        assert torch.equal(bits(y), bits(y2)) and torch.equal(bits(state), bits(other))
        _check(y, ry[:, t], my[:, t], k + (OPERAND[dt] if dt != "f32" else 0), f"token {t}")
    _check(state, rl, ml, k, "state")


@pytest.mark.parametrize("lengths", [None, [23, 9]])
def test_gradient_against_differences(lengths):
    """<gradient, v> against central differences of the 64-bit forward pass."""
    i = _inputs([9], 2, 23, 2, 12, 10, "f32", lengths=lengths)
    r = _backward(i, "differences")
    ins = {k: R.f64(i[k]) for k in NAMES}
    m = None if lengths is None else torch.tensor(lengths)
    f = lambda q, k, v, log_decay, state: A.attention(q, k, v, log_decay, i["scale"], state, m)
    mag = A.attention_backward(*_abs([A.wide(i["dy"])] + _args(i)), A.wide(i["dstate"]).abs())
    for name in NAMES:
        num, v = R.directional(f, ins, name, (R.f64(i["dy"]), R.f64(i["dstate"])))
        got = R.f64(getattr(r, name))
        bound = float(((R.EPS * got.abs() + (2 * 23 + 512) * R.EPS * mag[name].cpu()) * v.abs()).sum())
        assert abs(num - float((got * v).sum())) <= bound + 1e-6 * abs(num), name


def test_same_bits_on_every_call_and_nothing_past_the_outputs():
    i = _inputs([10], 2, 700, 3, 64, 96, "bf16", lengths=[700, 177])
    y0, s0 = _run(i)
    first = _back(i)
    need_f = cn.linear_attention_workspace_bytes(i["q"], i["v"])
    need = cn.linear_attention_workspace_bytes(i["q"], i["v"], backward=True, decay_grad=True)
    buf = torch.full((max(need, need_f) + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    out = torch.full((y0.numel() + 2048,), float("nan"), dtype=y0.dtype, device="cuda")
    for _ in range(3):
        y, s = _run(i, workspace=buf[:need_f], out=out[:y0.numel()].view(y0.shape))
        torch.cuda.synchronize()
        assert torch.equal(bits(y), bits(y0)) and torch.equal(bits(s), bits(s0))
        assert bool((buf[need_f:] == 0xA5).all()) and bool(torch.isnan(out[y0.numel():].float()).all())
        again = _back(i, workspace=buf[:need])
        torch.cuda.synchronize()
        assert all(torch.equal(bits(p), bits(q)) for p, q in zip(first, again))
        assert bool((buf[need:] == 0xA5).all())
        buf.fill_(0xA5)
    plain = _back(i, decay_grad=False)
    assert plain.log_decay is None
    assert all(torch.equal(bits(getattr(plain, k)), bits(getattr(first, k))) for k in ("q", "k", "v", "state"))
    with pytest.raises(cn.CnhwcError) as e:
        _back(i, workspace=buf[:need - 1])
    assert e.value.name == "WORKSPACE_TOO_SMALL"


def test_two_streams_at_once():
    """Calls queued on two streams give the bits that each gives alone."""
    ins = [_inputs([11, j], 1, 900, 3, 64, 64, "bf16") for j in range(2)]
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
    """A prompt, a token and a backward pass as one graph: every replay gives the eager bits."""
    i = _inputs([12], 1, 800, 2, 64, 64, "f16")
    tok = [i[k][:, 5].clone() for k in ("q", "k", "v")]

    def everything():
        y, s = _run(i)
        z = cn.linear_attention_step(*tok, i["log_decay"], s, scale=i["scale"])
        return (y, z, s, *_back(i))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        want = everything()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = everything()
    for _ in range(4):
        for t in got:
            t.zero_()
        graph.replay()
        everything()
        torch.cuda.synchronize()
        assert all(torch.equal(bits(p), bits(q)) for p, q in zip(got, want))


def test_empty_and_refusals():
    i = _inputs([13], 2, 5, 2, 8, 8, "f32")
    none = {k: (v[:, :0] if k in ("q", "k", "v", "dy") else v) for k, v in i.items()}
    y, last = _run(none)
    assert y.shape == (2, 0, 2, 8) and torch.equal(last, i["state"])
    r = _back(none)
    assert torch.equal(r.state, i["dstate"]) and not r.log_decay.any() and r.q.shape == (2, 0, 2, 8)
    run = lambda **kw: _run(dict(i, **kw))
    wide = torch.zeros(2, 5, 2, 257, device="cuda")
    for bad, kind in ((lambda: run(q=i["q"][0]), ValueError), (lambda: run(q=i["q"].cpu()), TypeError),
                      (lambda: run(k=i["k"].half()), TypeError), (lambda: run(k=i["k"][:, :4]), ValueError),
                      (lambda: run(v=i["v"][:, :, :1]), ValueError), (lambda: run(v=i["v"][0]), ValueError),
                      (lambda: run(q=i["q"].transpose(2, 3)), ValueError),
                      (lambda: run(log_decay=i["log_decay"][:1]), ValueError),
                      (lambda: run(log_decay=i["log_decay"].half()), TypeError),
                      (lambda: run(state=i["state"].half()), TypeError), (lambda: run(state=i["state"][:1]), ValueError),
                      (lambda: run(lengths=torch.zeros(2, dtype=torch.int64, device="cuda")), TypeError),
                      (lambda: run(q=wide, k=wide, state=None), cn.CnhwcError),
                      (lambda: run(v=wide, state=None), cn.CnhwcError),
                      (lambda: _run(i, out=i["v"]), cn.CnhwcError),
                      (lambda: cn.linear_attention_step(i["q"][:, 0], i["k"][:, 0], i["v"][:, 0], i["log_decay"], None),
                       ValueError),
                      (lambda: cn.linear_attention_backward(i["dy"][:1], i["q"], i["k"], i["v"], i["log_decay"]),
                       ValueError)):
        with pytest.raises(kind):
            bad()
