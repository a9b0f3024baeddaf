"""Linear attention where values are not finite, and what lies around the calls: an
infinity or NaN reaches the positions that see it and no other; other sequences,
heads and what is behind the outputs stay as they are."""
import numpy as np
import pytest
import torch

import attention_reference as A
import seq_reference as R
from gpu_util import bits

pytestmark = pytest.mark.gpu

cn = pytest.importorskip("convolution_nhwc_conv2d_amd")

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
# as in test_gpu_linear_attention.py: 2 L + 512 fp32 roundings, one rounding of an operand
OPERAND = {"f32": 0, "f16": 1 << 13, "bf16": 1 << 16}
L, AT = 100, 45


def _inputs(seed, dt, dk=48, dv=40):
    g = np.random.default_rng(seed)
    r = lambda *sh: R.rand(g, *sh).to(DT[dt]).cuda()
    return dict(q=r(2, L, 3, dk), k=r(2, L, 3, dk), v=r(2, L, 3, dv), dy=r(2, L, 3, dv),
                log_decay=-torch.tensor([0.01, 0.3, 0.0], device="cuda"))


def _near(got, ref, mag, dt, where):
    R.check(got, ref.cpu(), mag.cpu(), 2 * L + 512 + OPERAND[dt], where)


def _reference(i):
    a = [A.wide(i[k]) for k in ("q", "k", "v", "log_decay")]
    mag = [t.abs() for t in a[:3]] + [a[3]]
    return A.attention(*a, 0.2, None, None)[0], A.attention(*mag, 0.2, None, None)[0]


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("name", ["q", "k", "v"])
def test_what_is_not_finite_reaches_what_sees_it(name, bad, dt):
    """At one position and channel of one head of one sequence.  y before it, and of other
    heads and sequences, is the clean inputs'; of q it is that position's alone, of v that
    channel's alone."""
    i = _inputs([1], dt)
    ry, my = _reference(i)
    i[name] = i[name].clone()
    i[name][1, AT, 2, 7] = bad
    y, last = cn.linear_attention(i["q"], i["k"], i["v"], i["log_decay"], scale=0.2, return_state=True)
    hit = torch.zeros_like(y, dtype=torch.bool)
    if name == "q":
        hit[1, AT, 2] = True
    elif name == "k":
        hit[1, AT:, 2] = True
    else:
        hit[1, AT:, 2, 7] = True
    assert not torch.isfinite(y[hit]).any()
    clean = torch.where(hit, ry.to(y.dtype), y)
    _near(clean, ry, my, dt, f"{name} {bad}")
    state_hit = torch.zeros_like(last, dtype=torch.bool)
    if name == "k":
        state_hit[1, 2, 7] = True
    elif name == "v":
        state_hit[1, 2, :, 7] = True
    assert torch.isfinite(last[~state_hit]).all() and not torch.isfinite(last[state_hit]).any()


@pytest.mark.parametrize("dt", list(DT))
def test_gradients_beside_what_is_not_finite(dt):
    """dy not a number at one position: dq there alone, dk and dv there and before it."""
    i = _inputs([2], dt)
    run = lambda: cn.linear_attention_backward(i["dy"], i["q"], i["k"], i["v"], i["log_decay"], scale=0.2)
    clean = run()
    i["dy"] = i["dy"].clone()
    i["dy"][1, AT, 2, 7] = float("nan")
    r = run()
    for name in "qkv":
        got, was = getattr(r, name), getattr(clean, name)
        hit = torch.zeros_like(got, dtype=torch.bool)
        if name == "q":
            hit[1, AT, 2] = True
        elif name == "k":
            hit[1, :AT + 1, 2] = True
        else:
            hit[1, :AT + 1, 2, 7] = True
        assert torch.isnan(got[hit]).all(), name
        # the careful way adds in another order
        d = (got.double() - was.double())[~hit].norm() / was.double().norm()
        assert float(d) < (2.0 ** -20 if dt == "f32" else 4 * R.ROUND[DT[dt]]), name


@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_sizes_far_apart(dt):
    """Heads and channels whose values differ by large powers of two keep their digits:
    what brings f16's operands into range is of a row, a column or a head."""
    i = _inputs([3], dt)
    i["v"] = (i["v"].double() * torch.exp2(-(torch.arange(40, device="cuda") % 11).double())).to(DT[dt])
    i["k"] = (i["k"].double() * torch.tensor([1e-3, 1.0, 30.0], device="cuda").double()[:, None]).to(DT[dt])
    i["q"] = (i["q"].double() * torch.tensor([20.0, 1e-2, 1.0], device="cuda").double()[:, None]).to(DT[dt])
    y, last = cn.linear_attention(i["q"], i["k"], i["v"], i["log_decay"], scale=0.2, return_state=True)
    a = [A.wide(i[k]) for k in ("q", "k", "v", "log_decay")]
    ry, rl = A.attention(*a, 0.2, None, None)
    my, ml = A.attention(*[t.abs() for t in a[:3]], a[3], 0.2, None, None)
    _near(y, ry, my, dt, "y")
    R.check(last, rl.cpu(), ml.cpu(), 2 * L + 512, "state")


def test_rows_behind_the_outputs_and_no_channels():
    """out= inside a larger buffer: what is around it stays."""
    i = _inputs([4], "bf16")
    want = cn.linear_attention(i["q"], i["k"], i["v"], i["log_decay"])
    buf = torch.full((want.numel() + 8192,), float("nan"), dtype=want.dtype, device="cuda")
    out = buf[4096:4096 + want.numel()].view(want.shape)
    cn.linear_attention(i["q"], i["k"], i["v"], i["log_decay"], out=out,
                        lengths=torch.tensor([L, 3], dtype=torch.int32, device="cuda"))
    assert torch.equal(bits(out[0]), bits(want[0])) and not out[1, 3:].any()
    assert torch.isnan(buf[:4096]).all() and torch.isnan(buf[4096 + want.numel():]).all()
    none = torch.zeros(3, 0, device="cuda")
    for call in (lambda: cn.rms_norm(none, return_stats=True), lambda: cn.rms_norm_quantized(none),
                 lambda: cn.linear_attention(i["q"][..., :0], i["k"][..., :0], i["v"], i["log_decay"])):
        with pytest.raises((cn.CnhwcError, ValueError)):
            call()


def test_more_heads_than_a_launch_takes():
    z = torch.zeros(1, 1, 1, 1, device="cuda").expand(1, 1, (1 << 20) + 1, 1)
    with pytest.raises(cn.CnhwcError) as e:
        cn.linear_attention(z, z, z, torch.zeros((1 << 20) + 1, device="cuda"))
    assert e.value.name == "UNSUPPORTED"


def test_many_heads():
    """70000 sequences of two positions: more than fill the device at once."""
    n = 70000
    g = torch.Generator(device="cuda").manual_seed(5)
    q, k, v = (torch.randint(-2, 3, (n, 2, 1, 4), generator=g, device="cuda").half() for _ in range(3))
    y, s = cn.linear_attention(q, k, v, torch.zeros(1, device="cuda"), return_state=True)
    kv = (k[..., :, None] * v[..., None, :])[:, :, 0].float()
    assert torch.equal(s[:, 0], kv.sum(1))
    want = torch.stack([(q[:, t, 0, :, None].float() * kv[:, :t + 1].sum(1)).sum(1) for t in range(2)], 1)
    assert torch.equal(y[:, :, 0], want.half())


@pytest.mark.parametrize("dt", list(DT))
def test_growth_over_few_positions(dt):
    """Factors e^3 and e^1.5 a position, in sequences so short that every state fits
    float32, while the same growth over a whole chunk of positions does not."""
    i = _inputs([6], dt)
    n, l = 2, 3
    q, k, v, dy = (i[x][:, :l] for x in ("q", "k", "v", "dy"))
    growth = torch.tensor([3.0, 1.5, -1.0], device="cuda")
    lengths = torch.tensor([3, 2], dtype=torch.int32, device="cuda")
    y, last = cn.linear_attention(q, k, v, growth, scale=0.2, lengths=lengths, return_state=True)
    r = cn.linear_attention_backward(dy, q, k, v, growth, scale=0.2, lengths=lengths, decay_grad=True)
    a = [A.wide(t) for t in (q, k, v, growth)] + [0.2, None, lengths]
    mag = [t.abs() for t in a[:3]] + a[3:]
    want = A.attention(*a) + tuple(A.attention_backward(A.wide(dy), *a, None)[x] for x in ("q", "k", "v", "log_decay"))
    size = A.attention(*mag) + tuple(A.attention_backward(A.wide(dy).abs(), *mag, None)[x]
                                     for x in ("q", "k", "v", "log_decay"))
    # e^(3 d) of a product that is rounded, d <= 3: 9 more units, in both factors of a term
    units = 2 * l + 512 + 20
    for name, got, ref, m in zip(("y", "state", "dq", "dk", "dv", "dlog_decay"), (y, last, r.q, r.k, r.v, r.log_decay),
                                 want, size):
        R.check(got, ref.cpu(), m.cpu(), units + (0 if got.dtype == torch.float32 else OPERAND[dt]) + n * l, name)


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("dk,dv", [(128, 128), (72, 100), (40, 100), (100, 40), (130, 90)])
def test_heads_that_fill_the_device(dk, dv, dt):
    """130 heads, so that float32's passes take half as many columns a workgroup where there are
    more than 64; ragged, with states."""
    g = np.random.default_rng([7, dk, dv])
    n, l, h = 5, 70, 26
    r = lambda *sh: R.rand(g, *sh).cuda()
    q, k, v, dy = (r(n, l, h, d).to(DT[dt]) for d in (dk, dk, dv, dv))
    state, dstate = r(n, h, dk, dv).float(), r(n, h, dk, dv).float()
    decay = -torch.from_numpy(np.exp(g.uniform(-6, 0, h)).astype(np.float32)).cuda()
    lengths = torch.tensor([70, 0, 33, 64, 1], dtype=torch.int32, device="cuda")
    y, last = cn.linear_attention(q, k, v, decay, scale=0.1, state=state, lengths=lengths, return_state=True)
    b = cn.linear_attention_backward(dy, q, k, v, decay, scale=0.1, state=state, lengths=lengths, dstate=dstate,
                                     decay_grad=True)
    a = [A.wide(t) for t in (q, k, v, decay)] + [0.1, A.wide(state), lengths]
    mag = [t.abs() for t in a[:3]] + a[3:5] + [a[5].abs(), lengths]
    names = ("q", "k", "v", "log_decay", "state")
    ref, size = A.attention(*a), A.attention(*mag)
    back, bsize = A.attention_backward(A.wide(dy), *a, A.wide(dstate)), A.attention_backward(
        A.wide(dy).abs(), *mag, A.wide(dstate).abs())
    units = 2 * l + 512
    R.check(y, ref[0].cpu(), size[0].cpu(), units + OPERAND[dt], "y")
    R.check(last, ref[1].cpu(), size[1].cpu(), units, "state")
    for name, got in zip(names, b):
        more = n * l if name == "log_decay" else 0 if name == "state" else OPERAND[dt]
        R.check(got, back[name].cpu(), bsize[name].cpu(), units + more, "d" + name)
