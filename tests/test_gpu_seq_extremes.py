"""The sequence operators on values at the ends of their types."""
import numpy as np
import pytest
import torch

import seq_reference as R
from gpu_util import bits

pytestmark = pytest.mark.gpu

cn = pytest.importorskip("convolution_nhwc_conv2d_amd")

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def _large(dt):
    """100, 1e30 where the type holds it, and its largest value."""
    return [100.0] + ([] if dt == "f16" else [1e30]) + [torch.finfo(DT[dt]).max]


@pytest.mark.parametrize("dt", list(DT))
def test_conv_silu_of_large_values(dt):
    """One tap of 1: pre is x itself.  For x <= -100 silu and its slope are below
    2^-126, so 0 to the type; for x >= 100 they are x and 1 to its last place."""
    v = _large(dt)
    x = torch.tensor([-t for t in v] + v, dtype=torch.float64).to(DT[dt]).cuda()
    x = x.repeat(2, 5, 8)  # [2, 5, C]: vectors and, cut by one channel, single elements
    for c in (x.shape[2], x.shape[2] - 1):
        xc = x[..., :c].contiguous()
        w = torch.zeros(c, 4, dtype=xc.dtype, device="cuda")
        w[:, 3] = 1
        low = (xc < 0).cpu()
        tiny = R.TINY[xc.dtype]
        y = cn.causal_conv1d(xc, w, activation="silu")
        assert (R.f64(y)[low].abs() <= tiny).all() and torch.equal(y.cpu()[~low], xc.cpu()[~low])
        state = torch.zeros(2, 3, c, dtype=xc.dtype, device="cuda")
        assert torch.equal(bits(cn.causal_conv1d_step(xc[:, 0], state, w, activation="silu")), bits(y[:, 0]))
        dy = torch.full_like(xc, 2.0)
        r = cn.causal_conv1d_backward(dy, xc, w, torch.zeros(c, dtype=xc.dtype, device="cuda"), activation="silu")
        assert (R.f64(r.x)[low].abs() <= tiny).all() and (R.f64(r.x)[~low] == 2.0).all()
        assert torch.equal(R.f64(r.bias), (~low).double().sum((0, 1)) * 2.0)


def _gated(dt, s):
    """Channels with the large gates, half of them negative; products with the
    positive ones stay inside the type."""
    v = _large(dt)
    gates = torch.tensor(([-t for t in v] + v) * 8, dtype=torch.float64)
    d, n, l = len(gates), 2, 12
    g = np.random.default_rng([1, s])
    t = DT[dt]
    r = lambda *sh, dtype=t, **kw: R.rand(g, *sh, **kw).to(dtype).cuda()
    f = torch.float32
    low = gates < 0
    dy = R.rand(g, n, l, d) * torch.where(low, 4.0, 0.01)
    return dict(u=r(n, l, d), delta=r(n, l, d), a=-r(d, s, dtype=f).abs() - 0.05, b=r(n, l, s),
                c=r(n, l, s, scale=0.005), gate=gates.to(t).cuda().expand(n, l, d).contiguous(), dy=dy.to(t).cuda(),
                low=low)


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("s", [8, 16])
def test_scan_gates_of_large_values(s, dt):
    """The reference's magnitudes take silu of the gate, so a closed gate's bound is 2^-126."""
    i = _gated(dt, s)
    args = (i["u"], i["delta"], i["a"], i["b"], i["c"])
    y, last = cn.selective_scan(*args, gate=i["gate"], softplus=True, return_state=True)
    ref = [R.f64(t) for t in args] + [None, R.f64(i["gate"]), None, True, None, None]
    R.check(y, R.scan(*ref)[0], R.scan(*ref, absolute=True)[0], 16 * 12 + 64, "y")
    state = torch.zeros_like(last)
    tok = [t[:, 0] if t.dim() == 3 else t for t in args]
    assert torch.equal(bits(cn.selective_scan_step(*tok, state, gate=i["gate"][:, 0], softplus=True)), bits(y[:, 0]))


@pytest.mark.parametrize("dt", list(DT))
def test_nan_passes_silu(dt):
    """A gate or a pre-activation that is no number leaves none, in its own place alone."""
    i = _gated(dt, 8)
    gate = torch.ones_like(i["gate"])
    gate[0, 5, 3] = float("nan")
    args = (i["u"], i["delta"], i["a"], i["b"], i["c"])
    y = cn.selective_scan(*args, gate=gate, softplus=True)
    hit = torch.isnan(gate)
    assert torch.equal(torch.isnan(y), hit)
    r = cn.selective_scan_backward(i["dy"], *args, gate=gate, softplus=True)
    assert torch.equal(torch.isnan(r.gate), hit)
    assert torch.isnan(r.c[0, 5]).all() and not torch.isnan(r.c[0, 4]).any() and torch.isnan(r.u[0, 5, 3])
    x = torch.ones(2, 9, 16, dtype=DT[dt], device="cuda")
    x[1, 4, 6] = float("nan")
    w = torch.ones(16, 2, dtype=DT[dt], device="cuda")
    y = cn.causal_conv1d(x, w, activation="silu")
    assert torch.equal(torch.isnan(y).nonzero(), torch.tensor([[1, 4, 6], [1, 5, 6]], device="cuda"))
    r = cn.causal_conv1d_backward(torch.ones_like(x), x, w, activation="silu")
    assert torch.isnan(r.x[1, 3:6, 6]).all() and int(torch.isnan(r.x).sum()) == 3 and int(torch.isnan(r.w).sum()) == 2


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("s", [8, 16])
def test_scan_gradient_of_large_gates(s, dt):
    """Through a closed gate nothing comes back, whatever the gradient in front of
    it; the reference's magnitude of dgate grows with the gate, so that one is
    compared with 0 (|z silu'(z)| is below 2^-126 there) and with dy y."""
    i = _gated(dt, s)
    args = (i["u"], i["delta"], i["a"], i["b"], i["c"])
    r = cn.selective_scan_backward(i["dy"], *args, gate=i["gate"], softplus=True)
    ref = [R.f64(i["dy"])] + [R.f64(t) for t in args] + [None, R.f64(i["gate"]), None, True, None, None, None]
    want, mag = R.scan_backward(*ref), R.scan_backward(*ref, absolute=True)
    k = 32 * 12 + 128
    for name in ("u", "delta", "a", "b", "c"):
        R.check(getattr(r, name), want[name], mag[name], k + (2 * 12 if name == "a" else 0), "d" + name)
    low = i["low"]
    dgate = R.f64(r.gate)
    assert (dgate[..., low].abs() <= R.TINY[DT[dt]]).all()
    y = cn.selective_scan(*[t.float() for t in args], softplus=True)  # without the gate
    dyy = R.f64(i["dy"]) * R.f64(y)
    bound = (R.ROUND[DT[dt]] + 2 * k * R.EPS) * dyy.abs() + k * R.EPS * R.f64(i["dy"]).abs() * R.scan(
        *ref[1:6], None, None, None, True, None, None, absolute=True)[0] + R.TINY[DT[dt]]
    assert ((dgate - dyy).abs() <= bound)[..., ~low].all()


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("s", [5, 16, 32])
def test_scan_rates_without_end(s, dt):
    """a of minus infinity (and of the lowest float): the state holds the newest
    position alone, and past the lengths it stands still.  The reference of the
    gradient takes -1e30, whose decay is the same 0 and whose products are finite."""
    g = np.random.default_rng([2, s])
    n, l, d = 3, 21, 40
    t = DT[dt]
    r = lambda *sh, dtype=t, **kw: R.rand(g, *sh, **kw).to(dtype).cuda()
    f = torch.float32
    i = dict(u=r(n, l, d), delta=r(n, l, d), a=-r(d, s, dtype=f).abs() - 0.05, b=r(n, l, s), c=r(n, l, s))
    finite = i["a"].clone()
    i["a"][::2, ::2], finite[::2, ::2] = -float("inf"), -1e30
    i["a"][1::4, 1::2], finite[1::4, 1::2] = torch.finfo(f).min, -1e30
    lengths = torch.tensor([21, 6, 0], dtype=torch.int32, device="cuda")
    state, dy, dstate = r(n, d, s, dtype=f), r(n, l, d), r(n, d, s, dtype=f)
    y, last = cn.selective_scan(*i.values(), softplus=True, state=state, lengths=lengths, return_state=True)
    ref = [R.f64(v) for v in dict(i, a=finite).values()] + [None, None, None, True, R.f64(state), lengths]
    for got, want, mag in zip((y, last), R.scan(*ref), R.scan(*ref, absolute=True)):
        R.check(got, want, mag, 16 * l + 64, "forward")
    assert torch.equal(last[2], state[2])
    tok = [v[:, 0] if v.dim() == 3 else v for v in i.values()]
    moved = state.clone()
    y0 = cn.selective_scan_step(*tok, moved, softplus=True)
    y1, s1 = cn.selective_scan(*[v[:, :1] if v.dim() == 3 else v for v in i.values()], softplus=True, state=state,
                               return_state=True)
    assert torch.equal(bits(y0), bits(y1[:, 0])) and torch.equal(bits(moved), bits(s1))
    grads = cn.selective_scan_backward(dy, *i.values(), softplus=True, state=state, lengths=lengths, dstate=dstate)
    args = [R.f64(dy)] + ref + [R.f64(dstate)]
    want, mag = R.scan_backward(*args), R.scan_backward(*args, absolute=True)
    for name in ("u", "delta", "a", "b", "c", "state"):
        R.check(getattr(grads, name), want[name], mag[name], 32 * l + 128 + (n * l if name == "a" else 0), "d" + name)


@pytest.mark.parametrize("dt", list(DT))
def test_norm_of_constant_rows(dt):
    """A constant row has that constant as its mean and no variance, whatever its
    width: y is the bias, and rstd 1 / sqrt(eps).  In 16 bits the sums of these
    rows are exact.  In 32 the sum's rounding, up to some 80 units of the mean's
    last place, is exactly what is left of each element, and so is taken out;
    what stays in the variance of it is 2^-16 of its square."""
    eps = 1e-5
    for c in [32, 33, 96, 100, 480, 513, 1000, 1056, 1999, 2048, 2560, 4097, 5000, 7168, 8192, 9001, 17000, 33000, 66000]:
        v = torch.tensor([3000.0, 7.25, 3000.1, -0.1, 1e-3, 12345.678, 0.0])
        x = v[:, None].expand(len(v), c).to(DT[dt]).cuda().contiguous()
        g = np.random.default_rng([4, c])
        w, b = (R.rand(g, c).to(DT[dt]).cuda() for _ in range(2))
        y, mean, rstd = cn.layer_norm(x, w, b, eps, return_stats=True)
        assert torch.equal(mean, x[:, 0].float()), c
        assert torch.equal(y, b.expand(len(v), c)), c
        left = 2.0 ** -16 * (80 * R.EPS * x[:, 0].double().cpu()) ** 2
        assert ((R.f64(rstd) - eps ** -0.5).abs() <= eps ** -0.5 * (left / eps + 8 * R.EPS)).all(), c
        assert torch.equal(cn.layer_norm(x, eps=eps), torch.zeros_like(x)), c


def test_norm_mean_of_infinity():
    """The mean of a row with an infinity is that infinity."""
    x = torch.ones(2, 300, device="cuda")
    x[0, 7], x[1, 9] = float("inf"), -float("inf")
    _, mean, _ = cn.layer_norm(x, return_stats=True)
    assert mean.tolist() == [float("inf"), -float("inf")]
