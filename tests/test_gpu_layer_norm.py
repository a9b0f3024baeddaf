"""Layer norm on the GPU against the 64-bit reference, element by element.

The bound's k (32-bit roundings that can add up): a thread sums at most 64
elements of a row one after the other and the tree adds 10 (the mean, then the
variance, then their effect on y): 256.  The parameter gradients add the rows.
"""
import numpy as np
import pytest
import torch

import seq_reference as R
from gpu_util import bits

pytestmark = pytest.mark.gpu

cn = pytest.importorskip("convolution_nhwc_conv2d_amd")

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
K = 256
# every register tile and the ones past them, whole and ragged, vectors and single elements
WIDTHS = [1, 2, 7, 8, 24, 33, 64, 100, 127, 130, 257, 512, 513, 1000, 1024, 2048, 2056, 4096, 5000, 8192, 12288, 16384,
          17000, 33000, 66000]


def _params(g, c, dt, param):
    pt = DT[dt] if param == "same" else torch.float32
    return R.rand(g, c, scale=0.2, shift=1.0).to(pt).cuda(), R.rand(g, c, scale=0.2).to(pt).cuda()


def _forward(x, w, b, where):
    y, mean, rstd = cn.layer_norm(x, w, b, 1e-5, return_stats=True)
    ry, rm, rr, mag = R.layer_norm(R.f64(x), R.f64(w), R.f64(b), 1e-5)
    R.check(y, ry, mag, K, where + " y")
    R.check(mean, rm, R.f64(x).abs().mean(-1), K, where + " mean")
    var_mag = 1 + (R.f64(x).square().mean(-1)) * rr * rr  # the row's square against its variance
    R.check(rstd, rr, rr * var_mag, K, where + " rstd")
    return y, mean, rstd


def _backward(dy, x, mean, rstd, w, where):
    dx, dw, db = cn.layer_norm_backward(dy, x, mean, rstd, w)
    args = [R.f64(t) for t in (dy, x, mean, rstd, w)]
    want, mag = R.layer_norm_backward(*args), R.layer_norm_backward(*args, absolute=True)
    rows = x.numel() // x.shape[-1]
    R.check(dx, want[0], mag[0], K, where + " dx")
    if w is None:
        assert dw is None and db is None
        return dx, dw, db
    R.check(dw, want[1], mag[1], K + rows, where + " dw")
    R.check(db, want[2], mag[2], K + rows, where + " db")
    return dx, dw, db


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("c", WIDTHS)
def test_widths(c, dt):
    g = np.random.default_rng([1, c])
    rows = 5 if c > 4096 else 37
    x = R.rand(g, rows, c, scale=1.5, shift=0.5).to(DT[dt]).cuda()
    w, b = _params(g, c, dt, "same")
    _, mean, rstd = _forward(x, w, b, f"{dt} {c}")
    _backward(R.rand(g, rows, c).to(DT[dt]).cuda(), x, mean, rstd, w, f"{dt} {c}")


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("rows", [1, 2, 3, 63, 700, 4097])
def test_row_counts(rows, dt):
    g = np.random.default_rng([2, rows])
    for c in (40, 192):
        x = R.rand(g, rows, c).to(DT[dt]).cuda()
        w, b = _params(g, c, dt, "same")
        _, mean, rstd = _forward(x, w, b, f"{rows}x{c}")
        _backward(R.rand(g, rows, c).to(DT[dt]).cuda(), x, mean, rstd, w, f"{rows}x{c}")


@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_float32_parameters(dt):
    g = np.random.default_rng(3)
    x = R.rand(g, 50, 264).to(DT[dt]).cuda()
    w, b = _params(g, 264, dt, "f32")
    y, mean, rstd = _forward(x, w, b, dt)
    _, dw, db = _backward(R.rand(g, 50, 264).to(DT[dt]).cuda(), x, mean, rstd, w, dt)
    assert dw.dtype == db.dtype == torch.float32 and y.dtype == DT[dt]


def test_without_parameters_and_without_bias():
    g = np.random.default_rng(4)
    x, dy = (R.rand(g, 9, 72).half().cuda() for _ in range(2))
    w, _ = _params(g, 72, "f16", "same")
    _, mean, rstd = _forward(x, None, None, "plain")
    _backward(dy, x, mean, rstd, None, "plain")
    _forward(x, w, None, "no bias")


@pytest.mark.parametrize("dt", list(DT))
def test_strided_and_unaligned_rows(dt):
    """Slices of wider rows, of every second row, at odd element offsets, and a broadcast gradient."""
    g = np.random.default_rng(5)
    big = R.rand(g, 3, 22, 400).to(DT[dt]).cuda()
    w, b = _params(g, 96, dt, "same")
    for name, x in (("half", big[..., 96:192]), ("rows", big[:, ::2, :96]), ("odd", big[..., 5:101]),
                    ("last", big[:, -1, 16:112])):
        _, mean, rstd = _forward(x, w, b, name)
        _backward(R.rand(g, *x.shape).to(DT[dt]).cuda(), x, mean, rstd, w, name)
        dy = R.rand(g, 96).to(DT[dt]).cuda().expand(x.shape)  # strides of 0
        _backward(dy, x, mean, rstd, w, name + " broadcast")
    w4 = w.clone()
    x4 = big[:, :, :384].reshape(3, 2, 11, 384)[..., :96]
    y4 = cn.layer_norm(x4, w4, b)
    assert torch.equal(bits(y4), bits(cn.layer_norm(x4.contiguous(), w4, b)))


def test_offsets_past_32_bits():
    """Two rows more than 2^31 elements apart."""
    far = (1 << 31) + 64
    buf = torch.empty(far + 256, dtype=torch.bfloat16, device="cuda")
    x = buf.as_strided((2, 128), (far, 1))
    g = np.random.default_rng(6)
    x.copy_(R.rand(g, 2, 128).bfloat16().cuda())
    w, b = _params(g, 128, "bf16", "same")
    _, mean, rstd = _forward(x, w, b, "far")
    _backward(x, x, mean, rstd, w, "far")


def test_large_mean_and_constant_rows():
    """The variance is not the difference of two large sums; a constant row gives the bias."""
    g = np.random.default_rng(7)
    x = (R.rand(g, 6, 300) + 3000.0).cuda()
    x[2] = 7.25
    w, b = _params(g, 300, "f32", "same")
    y, _, rstd = _forward(x, w, b, "mean 3000")
    assert torch.equal(y[2], b) and abs(float(rstd[2]) - 1e5 ** 0.5) < 1e-2


def test_infinity_and_nan_stay_in_their_rows():
    g = np.random.default_rng(8)
    x = R.rand(g, 12, 136).cuda()
    clean = cn.layer_norm(x)
    x[3, 5], x[7, 9] = float("inf"), float("nan")
    y = cn.layer_norm(x)
    assert torch.isnan(y[3]).all() and torch.isnan(y[7]).all()
    keep = [i for i in range(12) if i not in (3, 7)]
    assert torch.equal(y[keep], clean[keep])


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_gradient_against_differences(dt):
    """<dx, v> and <dw, v> against central differences of the 64-bit forward pass.
    The values differ by the gradient's own bound, summed over the direction."""
    g = np.random.default_rng(9)
    x, dy = (R.rand(g, 11, 80).to(DT[dt]).cuda() for _ in range(2))
    w, b = _params(g, 80, dt, "same")
    _, mean, rstd = cn.layer_norm(x, w, b, return_stats=True)
    dx, dw, db = (R.f64(t) for t in cn.layer_norm_backward(dy, x, mean, rstd, w))
    f = lambda x, w, b: R.layer_norm(x, w, b, 1e-5)[:1]
    ins = dict(x=R.f64(x), w=R.f64(w), b=R.f64(b))
    args = [R.f64(t) for t in (dy, x, mean, rstd, w)]
    mags = dict(zip("xwb", R.layer_norm_backward(*args, absolute=True)))
    for name, got in (("x", dx), ("w", dw), ("b", db)):
        num, v = R.directional(f, ins, name, (R.f64(dy),))
        bound = float(((R.ROUND[DT[dt]] * got.abs() + (K + 11) * R.EPS * mags[name]) * v.abs()).sum())
        assert abs(num - float((got * v).sum())) <= bound + 1e-7 * abs(num), name


def test_same_bits_on_every_call_and_nothing_past_the_outputs():
    g = np.random.default_rng(10)
    x, dy = (R.rand(g, 1500, 264).bfloat16().cuda() for _ in range(2))
    w, b = _params(g, 264, "bf16", "same")
    y0, mean, rstd = cn.layer_norm(x, w, b, return_stats=True)
    first = cn.layer_norm_backward(dy, x, mean, rstd, w)
    need = cn.layer_norm_backward_workspace_bytes(x, w)
    assert need > 0
    buf = torch.full((need + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    out = torch.full((y0.numel() + 2048,), float("nan"), dtype=x.dtype, device="cuda")
    for _ in range(3):
        y = cn.layer_norm(x, w, b, out=out[:y0.numel()].view(y0.shape))
        again = cn.layer_norm_backward(dy, x, mean, rstd, w, workspace=buf[:need])
        torch.cuda.synchronize()
        assert torch.equal(bits(y), bits(y0))
        assert all(torch.equal(bits(p), bits(q)) for p, q in zip(first, again))
        assert bool((buf[need:] == 0xA5).all()) and bool(torch.isnan(out[y0.numel():].float()).all())
    with pytest.raises(cn.CnhwcError) as e:
        cn.layer_norm_backward(dy, x, mean, rstd, w, workspace=buf[:need - 1])
    assert e.value.name == "WORKSPACE_TOO_SMALL"


def test_empty_and_refusals():
    x = torch.zeros(0, 5, 16, device="cuda")
    w = torch.ones(16, device="cuda")
    y, mean, rstd = cn.layer_norm(x, w, w, return_stats=True)
    assert y.shape == x.shape and mean.shape == (0, 5)
    dx, dw, db = cn.layer_norm_backward(x, x, mean, rstd, w)
    assert dx.shape == x.shape and not dw.any() and not db.any()
    x = torch.zeros(4, 16, device="cuda")
    st = torch.zeros(4, device="cuda")
    for bad, kind in ((lambda: cn.layer_norm(x.cpu()), TypeError), (lambda: cn.layer_norm(x.double()), TypeError),
                      (lambda: cn.layer_norm(x.int()), TypeError), (lambda: cn.layer_norm(x, w[:8]), ValueError),
                      (lambda: cn.layer_norm(x, w.half()), TypeError), (lambda: cn.layer_norm(x, None, w), ValueError),
                      (lambda: cn.layer_norm(x.t()), ValueError), (lambda: cn.layer_norm(x, w, w, -1.0), cn.CnhwcError),
                      (lambda: cn.layer_norm(x, w, w, float("nan")), cn.CnhwcError),
                      (lambda: cn.layer_norm(x, out=x), cn.CnhwcError),
                      (lambda: cn.layer_norm(x, out=x.half()), TypeError),
                      (lambda: cn.layer_norm_backward(x[:3], x, st, st, w), ValueError),
                      (lambda: cn.layer_norm_backward(x, x, st.double(), st, w), TypeError),
                      (lambda: cn.layer_norm_backward(x, x, st[:2], st, w), ValueError)):
        with pytest.raises(kind):
            bad()
