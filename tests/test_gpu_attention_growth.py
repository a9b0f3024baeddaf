"""Linear attention's states under decays that leave fp32's ordinary range: infinite states; growth (log_decay
> 0) where the states themselves fit float32; and the digits that fast decays leave."""
import numpy as np
import pytest
import torch

import attention_reference as A
import seq_reference as R

pytestmark = pytest.mark.gpu

cn = pytest.importorskip("convolution_nhwc_conv2d_amd")

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
# as in test_gpu_linear_attention.py: one rounding of an operand
OPERAND = {"f32": 0, "f16": 1 << 13, "bf16": 1 << 16}


def _rows(seed, dt, n, l, h, dk, dv):
    g = np.random.default_rng(seed)
    r = lambda *sh: R.rand(g, *sh).to(DT[dt]).cuda()
    return r(n, l, h, dk), r(n, l, h, dk), r(n, l, h, dv), r(n, l, h, dv)


@pytest.mark.parametrize("dt", list(DT))
def test_an_infinite_state_stays_infinite(dt):
    """Through a token and through the runs of a prompt alike, and only where it is: each decay
    (of a token, of a chunk and of a run) is e^-0.5 or faster and no underflow."""
    q, k, v, _ = _rows([1], dt, 1, 700, 2, 64, 64)
    state = torch.zeros(1, 2, 64, 64, device="cuda")
    state[0, 1, 3, 5], state[0, 0, 60, 63] = float("inf"), float("-inf")
    hit = torch.isinf(state)
    was = state.clone()
    cn.linear_attention_step(q[:, 0], k[:, 0], v[:, 0], torch.tensor([-0.5, -1.0], device="cuda"), state)
    assert torch.equal(state[hit], was[hit]) and torch.isfinite(state[~hit]).all()
    assert cn.linear_attention_workspace_bytes(q, v) > 0  # more than one run
    _, last = cn.linear_attention(q, k, v, torch.tensor([-0.02, -0.05], device="cuda"), state=was, return_state=True)
    assert torch.equal(last[hit], was[hit]) and torch.isfinite(last[~hit]).all()


def _growing(dt, n, l, h, growth, late, early, seed):
    """The forward pass and the gradients that go through the state, with k and v only in the last
    `late` positions, and the gradients that go through its derivative, with q and dy only in
    the first `early` ones: every state is 0 or grows over that many positions."""
    q, k, v, dy = _rows(seed, dt, n, l, h, 64, 48)
    scale = 2.0 ** -int(growth * (late - 1) / np.log(2))  # y stays within f16
    g = torch.full((h,), growth, device="cuda")
    # 2 L + 512; each decay's exponent, g times positions, is rounded to 2^-24 of itself: at most
    # g late units more a factor, twice where two factors meet
    units = 2 * l + 512 + int(2 * growth * max(late, early))
    kl, vl, dl = k.clone(), v.clone(), dy.clone()
    kl[:, :l - late] = 0
    vl[:, :l - late] = 0
    dl[:, :l - late] = 0
    check = lambda got, ref, mag, name: R.check(got, ref.cpu(), mag.cpu(), units + (
        0 if got.dtype == torch.float32 else OPERAND[dt]) + (n * l if name == "dlog_decay" else 0), f"{name} {growth}")
    # k alone, v alone, and both: what is 0 in one of them leaves no state either
    for name, kk, vv in (("both", kl, vl), ("v everywhere", kl, v), ("k everywhere", k, vl)):
        y, last = cn.linear_attention(q, kk, vv, g, scale=scale, return_state=True)
        a = [A.wide(t) for t in (q, kk, vv, g)] + [scale, None, None]
        mag = [t.abs() for t in a[:3]] + a[3:]
        for t, ref, m, what in zip((y, last), A.attention(*a), A.attention(*mag), ("y", "state")):
            check(t, ref, m, f"{name}: {what}")
    r = cn.linear_attention_backward(dl, q, kl, v, g, scale=scale, decay_grad=True)
    a = [A.wide(t) for t in (dl, q, kl, v, g)] + [scale, None, None, None]
    mag = [t.abs() for t in a[:4]] + a[4:]
    want, size = A.attention_backward(*a), A.attention_backward(*mag)
    check(r.q, want["q"], size["q"], "dq")
    check(r.log_decay, want["log_decay"], size["log_decay"], "dlog_decay")
    qe, de, none = q.clone(), dy.clone(), torch.zeros_like(k)
    qe[:, early:] = 0
    de[:, early:] = 0
    state = torch.zeros(n, h, 64, 48, device="cuda")
    for name, qq, dd in (("both", qe, de), ("dy everywhere", qe, dy), ("q everywhere", q, de)):
        for kk, vv in ((k, torch.zeros_like(v)), (none, v)):
            r = cn.linear_attention_backward(dd, qq, kk, vv, g, scale=scale, state=state)
            a = [A.wide(t) for t in (dd, qq, kk, vv, g)] + [scale, A.wide(state), None, None]
            mag = [t.abs() for t in a[:4]] + a[4:]
            want, size = A.attention_backward(*a), A.attention_backward(*mag)
            for x in ("k", "v", "state"):
                check(getattr(r, x), want[x], size[x], f"{name}: d{x}")


@pytest.mark.parametrize("dt", list(DT))
def test_growth_over_many_runs(dt):
    """e^0.95 a position: a run of 96 positions or more grows by e^91, past float32; what grows
    starts 60 positions from the end."""
    n, l, h, growth = 1, 1200, 16, 0.95
    q = torch.empty(n, l, h, 64, dtype=DT[dt], device="cuda")
    runs = 1 + cn.linear_attention_workspace_bytes(q, q[..., :48]) // (n * h * 64 * 64 * 4)
    run = -(-(l // 32) // runs) * 32
    assert runs > 2 and growth * run > 89
    _growing(dt, n, l, h, growth, 60, 60, [2])


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("growth,l,late", [(1.4, 64, 20), (3.0, 30, 3), (5.0, 100, 3), (12.0, 70, 2), (44.0, 45, 1),
                                           (80.0, 33, 1), (1.5, 200, 9)])
def test_growth_within_a_chunk(growth, l, late, dt):
    """A chunk of 32 positions (of 64 for the decay's gradient) grows past float32."""
    _growing(dt, 2, l, 3, growth, late, min(late, 5), [3, l, late])


@pytest.mark.parametrize("dt", list(DT))
def test_growth_of_a_zero_state_over_a_whole_sequence(dt):
    """e^90 over 30 positions is past float32; nothing enters the state before the last one."""
    q, k, v, dy = _rows([4], dt, 1, 30, 1, 32, 32)
    k[:, :29] = 0
    g = torch.tensor([3.0], device="cuda")
    y, last = cn.linear_attention(q, k, v, g, state=torch.zeros(1, 1, 32, 32, device="cuda"), return_state=True)
    a = [A.wide(t) for t in (q, k, v, g)] + [1.0, None, None]
    mag = [t.abs() for t in a[:3]] + a[3:]
    for t, ref, m, units in zip((y, last), A.attention(*a), A.attention(*mag), (OPERAND[dt], 0)):
        R.check(t, ref.cpu(), m.cpu(), 2 * 30 + 512 + units, "growth of 0")


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("place", [0, 4, 5])
def test_growth_of_ragged_sequences(place, dt):
    """Steps of a few positions, in both directions, with lengths that end inside and on them, states
    from outside, rows behind the lengths, and rows off 16 bytes."""
    n, l, h, dk, dv = 4, 70, 3, 48, 40
    growth = torch.tensor([3.0, 0.7, -1.0], device="cuda")
    lengths = torch.tensor([20, 7, 0, 16], dtype=torch.int32, device="cuda")
    scale = 2.0 ** -86  # e^-60
    q, k, v, dy = _rows([6], dt, n, l, h, dk, dv)[:3] + (_rows([7], dt, n, l, h, dk, dv)[3],)

    def placed(t):
        buf = torch.full((n, l, h * t.shape[-1] + 12), float("nan"), dtype=t.dtype, device="cuda")
        x = buf[..., place:place + h * t.shape[-1]].unflatten(-1, (h, t.shape[-1]))
        x.copy_(t)
        for j, m in enumerate(lengths.tolist()):
            x[j, m:] = float("nan")
        return x
    q, k, v, dy = (placed(t) for t in (q, k, v, dy))
    g = np.random.default_rng(8)
    state, dstate = R.rand(g, n, h, dk, dv).cuda(), R.rand(g, n, h, dk, dv).cuda() * scale
    y, last = cn.linear_attention(q, k, v, growth, scale=scale, state=state, lengths=lengths, return_state=True)
    r = cn.linear_attention_backward(dy, q, k, v, growth, scale=scale, state=state, lengths=lengths, dstate=dstate,
                                     decay_grad=True)
    q, k, v, dy = (torch.nan_to_num(t) for t in (q, k, v, dy))
    a = [A.wide(t) for t in (q, k, v, growth)] + [scale, A.wide(state), lengths]
    mag = A.absolute(*a)
    mag[3] = a[3]
    want, size = A.attention(*a), A.attention(*mag)
    back = A.attention_backward(A.wide(dy), *a, A.wide(dstate))
    bsize = A.attention_backward(A.wide(dy).abs(), *mag, A.wide(dstate).abs())
    units = 2 * l + 512 + 2 * 3 * 20  # and the exponents' roundings, as in _growing
    for name, got, ref, m in [("y", y, want[0], size[0]), ("last", last, want[1], size[1])] + [
            (x, getattr(r, x), back[x], bsize[x]) for x in ("q", "k", "v", "log_decay", "state")]:
        more = n * l if name == "log_decay" else 0 if name in ("last", "state") else OPERAND[dt]
        R.check(got, ref.cpu(), m.cpu(), units + more, f"{name} {place}")
        if name in ("y", "q", "k", "v"):
            for j, x in enumerate(lengths.tolist()):
                assert not got[j, x:].any()
    assert torch.equal(last[2], state[2]) and torch.equal(r.state[2], dstate[2])


@pytest.mark.parametrize("dt", list(DT))
def test_digits_of_what_a_fast_decay_leaves(dt):
    """Keys of one channel each, so that a row of the state is one position's v under its decay,
    down to e^-31 of the last one's.  In f16, whose products have a narrow range, to 2^-50
    of the largest of a chunk's column, 2^-39 where the decay across a chunk is slower than 2^-8."""
    l, h = 32, 5
    _, _, v, dy = _rows([5], dt, 2, l, h, 32, 40)
    eye = torch.eye(l, dtype=DT[dt], device="cuda")[None, :, None].expand(2, l, h, l)
    g = -torch.tensor([0.2, 0.5, 0.7, 1.0, 0.17], device="cuda")
    least = torch.tensor([2.0 ** -50] * 4 + [2.0 ** -39], device="cuda").double()[:, None, None]

    def check(got, ref):
        tol = (2 * l + 512) * R.EPS * ref.abs() + 2.0 ** -126
        if dt == "f16":
            tol = tol + least * ref.abs().amax(2, keepdim=True)
        bad = (got.double() - ref).abs() > tol
        assert not bad.any(), torch.nonzero(bad)[0].tolist()
    _, last = cn.linear_attention(eye, eye, v, g, return_state=True)
    a = [A.wide(t) for t in (eye, eye, v, g)] + [1.0]
    check(last, A.attention(*a, None, None)[1])
    r = cn.linear_attention_backward(dy, eye, eye, v, g, state=torch.zeros_like(last))  # the gradient: from the end
    check(r.state, A.attention_backward(A.wide(dy), *a, A.wide(torch.zeros_like(last)), None, None)["state"])
