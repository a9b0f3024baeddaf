"""The root-mean-square norm on the GPU against the 64-bit reference, element by element.

The bound's k (32-bit roundings that can add up): a thread sums at most 64
squares of a row one after the other and the tree adds 10; the sum, the root and
the products add a few: 256.  The parameter's gradient adds the rows.  An
element in 8 bits is off its value by half a step, 2^-4 of it or, below 2^-6 of
the scale, 2^-10 of the scale.
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
K = 256
WIDTHS = [1, 2, 7, 8, 24, 33, 64, 100, 127, 130, 257, 512, 513, 1000, 1024, 2048, 2056, 4096, 5000, 8192, 12288, 16384,
          17000, 33000, 66000]


def _rand(g, shape, dt, **kw):
    return R.rand(g, *shape, **kw).to(DT[dt]).cuda()


def _forward(x, w, residual, where, eps=1e-6):
    r = cn.rms_norm(x, w, eps, residual=residual, return_stats=True)
    y, rstd = r[0], r[-1]
    ry, rz, rr, mag = A.rms_norm(*(R.f64(t) for t in (x, residual, w)), eps)
    R.check(y, ry, mag, K, where + " y")
    R.check(rstd, rr, 3 * rr, K, where + " rstd")
    if residual is None:
        assert len(r) == 2
        return y, x, rstd
    R.check(r[1], rz, rz.abs(), 1, where + " sum")
    return y, r[1], rstd


def _backward(dy, z, rstd, w, dsum, where):
    dx, dw = cn.rms_norm_backward(dy, z, rstd, w, dsum=dsum)
    args = [R.f64(t) for t in (dy, z, rstd, w, dsum)]
    want, mag = A.rms_norm_backward(*args), A.rms_norm_backward(*args, absolute=True)
    R.check(dx, want[0], mag[0], K, where + " dx")
    if w is None:
        assert dw is None
    else:
        R.check(dw, want[1], mag[1], K + z.numel() // z.shape[-1], where + " dw")
    return dx, dw


def _quantized(x, w, residual, group, where, eps=1e-6):
    r = cn.rms_norm_quantized(x, w, eps, group=group, residual=residual, return_stats=True)
    q, scale = r[0], r[1]
    ry, rz, rr, mag = A.rms_norm(*(R.f64(t) for t in (x, residual, w)), eps)
    assert q.dtype == torch.float8_e4m3fn and q.shape == x.shape and scale.dtype == torch.float32
    want = A.scales(ry, group)
    most = A.scales(mag, group)
    R.check(scale, want, most, K, where + " scale")
    s = R.f64(scale)
    s = (s[..., None] if not group else s.repeat_interleave(group, -1)).expand(ry.shape)
    got = q.cpu().float().double() * s
    assert torch.isfinite(got).all(), where
    half = torch.maximum(ry.abs() * 2.0 ** -4, s * 2.0 ** -10)
    off = (got - ry).abs()
    assert (off <= half * (1 + 2.0 ** -10) + 2 * K * R.EPS * mag).all(), f"{where}: {float((off - half).max())}"
    R.check(r[-1], rr, 3 * rr, K, where + " rstd")
    if residual is not None:
        R.check(r[2], rz, rz.abs(), 1, where + " sum")
    return r


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("c", WIDTHS)
def test_widths(c, dt):
    g = np.random.default_rng([1, c])
    rows = 5 if c > 4096 else 37
    x, res = _rand(g, (rows, c), dt, scale=1.5), _rand(g, (rows, c), dt, scale=3.0)
    w = _rand(g, (c,), dt, scale=0.2, shift=1.0)
    _forward(x, w, None, f"{dt} {c}")
    _, z, rstd = _forward(x, w, res, f"{dt} {c} residual")
    _backward(_rand(g, (rows, c), dt), z, rstd, w, _rand(g, (rows, c), dt), f"{dt} {c}")
    _quantized(x, w, res, None, f"{dt} {c} 8 bits")


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("groups", [1, 2, 3, 5, 8, 31, 64, 200, 600])
def test_groups(groups, group, dt):
    g = np.random.default_rng([2, groups, group])
    c, rows = groups * group, 3 if groups > 30 else 70
    # groups of very different sizes in one row
    x = R.rand(g, rows, groups, group) * torch.from_numpy(g.uniform(0.01, 4.0, (rows, groups, 1)).astype(np.float32))
    x = x.reshape(rows, c).to(DT[dt]).cuda()
    _quantized(x, _rand(g, (c,), dt, shift=1.0, scale=0.1), _rand(g, (rows, c), dt, scale=0.02), group, f"{c}/{group}")
    _quantized(x, None, None, group, f"{c}/{group} plain")


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("rows", [1, 2, 3, 63, 700, 4097])
def test_row_counts(rows, dt):
    g = np.random.default_rng([3, rows])
    for c in (40, 192):
        x, w = _rand(g, (rows, c), dt), _rand(g, (c,), dt, shift=1.0, scale=0.1)
        _, z, rstd = _forward(x, w, None, f"{rows}x{c}")
        _backward(_rand(g, (rows, c), dt), z, rstd, w, None, f"{rows}x{c}")
        _quantized(x, w, None, 64 if c == 192 else None, f"{rows}x{c}")


@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_float32_parameters_and_none(dt):
    g = np.random.default_rng(4)
    x, dy, w = _rand(g, (50, 264), dt), _rand(g, (50, 264), dt), _rand(g, (264,), "f32", shift=1.0, scale=0.2)
    y, _, rstd = _forward(x, w, None, dt)
    _, dw = _backward(dy, x, rstd, w, None, dt)
    assert dw.dtype == torch.float32 and y.dtype == DT[dt]
    _forward(x, None, dy, "no weight")
    _backward(dy, x, rstd, None, dy, "no weight")


@pytest.mark.parametrize("dt", list(DT))
def test_strided_and_unaligned_rows(dt):
    """Slices of wider rows, of every second row, at odd element offsets, broadcast rows."""
    g = np.random.default_rng(5)
    big, res = _rand(g, (3, 22, 400), dt), _rand(g, (3, 22, 400), dt)
    w = _rand(g, (128,), dt, scale=0.2, shift=1.0)
    for name, cut in (("half", lambda t: t[..., 128:256]), ("rows", lambda t: t[:, ::2, :128]),
                      ("odd", lambda t: t[..., 5:133]), ("last", lambda t: t[:, -1, 16:144])):
        x = cut(big)
        for other in (cut(res), res[:1, :1, 3:131].expand(x.shape) if x.dim() == 3 else res[0, :1, :128].expand(x.shape)):
            _, z, rstd = _forward(x, w, other, name)
            _backward(other, z, rstd, w, cut(res), name)
            _quantized(x, w, other, 32, name)
        _backward(x, x, cn.rms_norm(x, w, return_stats=True)[1], w, None, name)
    w1 = torch.cat([w, w])[1:129]  # a weight off its vectors
    _forward(big[..., :128], w1, res[..., :128], "weight")
    _quantized(big[..., :128], w1, None, 64, "weight")


def test_offsets_past_32_bits():
    far = (1 << 31) + 64
    buf = torch.empty(far + 256, dtype=torch.bfloat16, device="cuda")
    x = buf.as_strided((2, 128), (far, 1))
    g = np.random.default_rng(6)
    x.copy_(_rand(g, (2, 128), "bf16"))
    w = _rand(g, (128,), "bf16", shift=1.0, scale=0.2)
    _, z, rstd = _forward(x, w, x, "far")
    _backward(x, x, cn.rms_norm(x, w, return_stats=True)[1], w, x, "far")
    _quantized(x, w, x, 32, "far")


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("c", [96, 100, 2048, 70000])
def test_sum_in_place(c, dt):
    """sum_out on the residual: the bits of a sum of its own."""
    g = np.random.default_rng([7, c])
    x, res, w = _rand(g, (9, c), dt), _rand(g, (9, c), dt), _rand(g, (c,), dt)
    y, z = cn.rms_norm(x, w, residual=res)
    q, scale, z2 = cn.rms_norm_quantized(x, w, residual=res)
    a, b = res.clone(), res.clone()
    y1, z1 = cn.rms_norm(x, w, residual=a, sum_out=a)
    q1, scale1, z3 = cn.rms_norm_quantized(x, w, residual=b, sum_out=b)
    assert z1.data_ptr() == a.data_ptr() and z3.data_ptr() == b.data_ptr()
    for p, r in ((y, y1), (z, z1), (z, a), (z2, b), (z, z2), (scale, scale1)):
        assert torch.equal(bits(p), bits(r))
    assert torch.equal(q.view(torch.uint8), q1.view(torch.uint8))


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("group", [None, 32])
def test_ends_of_the_types(group, dt):
    """Rows of zeros, of the smallest values, and of infinity and NaN, which stay in their row or group."""
    g = np.random.default_rng(8)
    x = _rand(g, (6, 128), dt)
    x[1] = 0
    x[2] = torch.finfo(DT[dt]).tiny
    clean, cscale = cn.rms_norm_quantized(x, None, 1e-6, group=group)
    y = cn.rms_norm(x, None, 1e-6)
    assert not y[1].any() and not clean[1].float().any() and (cscale[1] == 2.0 ** -100).all()
    assert torch.isfinite(clean.float()).all() and torch.isfinite(cscale).all() and (cscale > 0).all()
    bad = x.clone()
    bad[3, 5], bad[4, 40] = float("inf"), float("nan")
    yb = cn.rms_norm(bad, None, 1e-6)
    assert torch.isnan(yb[3, 5]) and not yb[3, 6:].any() and torch.isnan(yb[4]).all()
    q, s = cn.rms_norm_quantized(bad, None, 1e-6, group=group)
    keep = [0, 1, 2, 5]
    assert torch.equal(q[keep].view(torch.uint8), clean[keep].view(torch.uint8)) and torch.equal(s[keep], cscale[keep])
    assert torch.isnan(q[3, 5].float()) and torch.isnan(q[4].float()).all()
    # an infinite weight: its row, or its group alone
    w = torch.ones(128, device="cuda").to(DT[dt])
    w[7] = float("inf")
    q, s = cn.rms_norm_quantized(x, w, 1e-6, group=group)
    v = q.float() * (s[..., None] if group is None else s.repeat_interleave(group, -1))
    assert torch.isnan(v[0, :32]).all() and (group is None or torch.isfinite(v[0, 32:]).all())


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_gradient_against_differences(dt):
    """<dx, v> and <dw, v> against central differences of the 64-bit forward pass."""
    g = np.random.default_rng(9)
    x, dy, ds = (_rand(g, (11, 80), dt) for _ in range(3))
    w = _rand(g, (80,), dt, shift=1.0, scale=0.2)
    _, rstd = cn.rms_norm(x, w, return_stats=True)
    dx, dw = (R.f64(t) for t in cn.rms_norm_backward(dy, x, rstd, w, dsum=ds))
    f = lambda x, w: A.rms_norm(x, None, w, 1e-6)[:2]
    ins = dict(x=R.f64(x), w=R.f64(w))
    mags = A.rms_norm_backward(*(R.f64(t) for t in (dy, x, rstd, w, ds)), absolute=True)
    for name, got, mag in (("x", dx, mags[0]), ("w", dw, mags[1])):
        num, v = R.directional(f, ins, name, (R.f64(dy), R.f64(ds)))
        bound = float(((R.ROUND[DT[dt]] * got.abs() + (K + 11) * R.EPS * mag) * v.abs()).sum())
        assert abs(num - float((got * v).sum())) <= bound + 1e-7 * abs(num), name


def test_same_bits_graphs_and_nothing_past_the_outputs():
    g = np.random.default_rng(10)
    x, dy, res = (_rand(g, (1500, 384), "bf16") for _ in range(3))
    w = _rand(g, (384,), "bf16")

    def everything(out=None, ws=None):
        r = cn.rms_norm(x, w, residual=res, return_stats=True, out=out)
        return (*r, *cn.rms_norm_quantized(x, w, group=128)[1:], *cn.rms_norm_backward(dy, r[1], r[2], w, dsum=res,
                                                                                       workspace=ws))
    first = everything()
    need = cn.rms_norm_backward_workspace_bytes(x, w)
    assert need > 0
    buf = torch.full((need + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    out = torch.full((x.numel() + 2048,), float("nan"), dtype=x.dtype, device="cuda")
    for _ in range(3):
        again = everything(out[:x.numel()].view(x.shape), buf[:need])
        torch.cuda.synchronize()
        assert all(torch.equal(bits(p), bits(q)) for p, q in zip(first, again))
        assert bool((buf[need:] == 0xA5).all()) and bool(torch.isnan(out[x.numel():].float()).all())
    with pytest.raises(cn.CnhwcError) as e:
        cn.rms_norm_backward(dy, x, first[2], w, workspace=buf[:need - 1])
    assert e.value.name == "WORKSPACE_TOO_SMALL"
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        everything()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = everything()
    for _ in range(3):
        for t in captured:
            t.zero_()
        graph.replay()
        everything()
        torch.cuda.synchronize()
        assert all(torch.equal(bits(p), bits(q)) for p, q in zip(first, captured))


def test_empty_and_refusals():
    x = torch.zeros(0, 5, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    y, z, rstd = cn.rms_norm(x, w, residual=x, return_stats=True)
    assert y.shape == z.shape == x.shape and rstd.shape == (0, 5)
    q, s = cn.rms_norm_quantized(x, w, group=32)
    assert q.shape == x.shape and s.shape == (0, 5, 2)
    dx, dw = cn.rms_norm_backward(x, x, rstd, w)
    assert dx.shape == x.shape and not dw.any()
    x = torch.zeros(4, 64, device="cuda")
    st = torch.zeros(4, device="cuda")
    for bad, kind in ((lambda: cn.rms_norm(x.cpu()), TypeError), (lambda: cn.rms_norm(x.double()), TypeError),
                      (lambda: cn.rms_norm(x, w[:8]), ValueError), (lambda: cn.rms_norm(x, w.half()), TypeError),
                      (lambda: cn.rms_norm(x.t()), ValueError), (lambda: cn.rms_norm(x, w, -1.0), cn.CnhwcError),
                      (lambda: cn.rms_norm(x, w, float("nan")), cn.CnhwcError),
                      (lambda: cn.rms_norm(x, out=x), cn.CnhwcError), (lambda: cn.rms_norm(x, out=x.half()), TypeError),
                      (lambda: cn.rms_norm(x, residual=x[:2]), ValueError),
                      (lambda: cn.rms_norm(x, residual=x.half()), TypeError),
                      (lambda: cn.rms_norm(x, sum_out=torch.empty_like(x)), ValueError),
                      (lambda: cn.rms_norm(x, residual=x + 1, sum_out=x), cn.CnhwcError),
                      (lambda: cn.rms_norm(x, residual=x[:1].expand(4, 64), sum_out=x[:1].expand(4, 64)), ValueError),
                      (lambda: cn.rms_norm_quantized(x, group=48), ValueError),
                      (lambda: cn.rms_norm_quantized(x, group=0), ValueError),
                      (lambda: cn.rms_norm_quantized(x, group=16), cn.CnhwcError),
                      (lambda: cn.rms_norm_quantized(x, out=x), TypeError),
                      (lambda: cn.rms_norm_quantized(x, group=32, scale_out=st), ValueError),
                      (lambda: cn.rms_norm_backward(x[:3], x, st, w), ValueError),
                      (lambda: cn.rms_norm_backward(x, x, st.double(), w), TypeError),
                      (lambda: cn.rms_norm_backward(x, x, st, w, dsum=x[:2]), ValueError)):
        with pytest.raises(kind):
            bad()
