"""Rotary positions on the GPU against the 64-bit reference, element by element.

The bound's k: sine and cosine are off by a few units of 2^-24 (their argument's
rounding, at most 0.79, and the series), the two products and the sum by one each: 12.
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
K = 12


def _rand(g, shape, dt):
    return R.rand(g, *shape).to(DT[dt]).cuda()


def _check(x, freqs, where, positions=None, offset=0, interleaved=False, scale=1.0, **kw):
    n, l = (x.shape[0], 1) if x.dim() == 3 else x.shape[:2]
    at = torch.arange(l) if positions is None else positions.cpu().long()
    at = (at[:, None] if x.dim() == 3 and positions is not None else at).expand(n, l) + offset
    args = dict(positions=positions, offset=offset, interleaved=interleaved, scale=scale)
    for f, sign in ((cn.rotary, 1), (cn.rotary_backward, -1)):
        y = f(x, freqs, **args, **kw)
        ref, mag = A.rotary(R.f64(x).reshape(n, l, *x.shape[-2:]), freqs.cpu(), at, interleaved, scale, sign)
        R.check(y.reshape(n, l, *x.shape[-2:]), ref, mag, K, where)
        r = 2 * freqs.shape[0]
        assert torch.equal(bits(y[..., r:]), bits(x[..., r:]))
    return y


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("d,r", [(1, 0), (2, 2), (3, 2), (8, 8), (16, 8), (34, 12), (64, 64), (64, 32), (80, 80),
                                 (96, 48), (100, 36), (128, 128), (128, 64), (128, 2), (256, 256), (250, 250)])
def test_sizes(d, r, interleaved, dt):
    g = np.random.default_rng([1, d, r])
    for n, l, h in ((2, 19, 3), (1, 1, 1), (1, 70, 9)):
        x = _rand(g, (n, l, h, d), dt)
        _check(x, cn.rotary_frequencies(r), f"{n}x{l}x{h}x{d}/{r}", interleaved=interleaved, scale=1.25)


@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("h", [1, 2, 3, 4, 5, 8, 17, 40, 130])
def test_heads_and_tokens(h, interleaved):
    g = np.random.default_rng([2, h])
    f = cn.rotary_frequencies(64)
    pos = torch.from_numpy(g.integers(0, 1 << 20, 33).astype(np.int32)).cuda()
    _check(_rand(g, (33, h, 128), "bf16"), f, f"{h} heads", positions=pos, interleaved=interleaved)
    _check(_rand(g, (33, h, 64), "f32"), f, f"{h} heads", positions=pos, interleaved=interleaved)
    _check(_rand(g, (33, h, 64), "f16"), f, f"{h} heads", offset=5, interleaved=interleaved)


def test_positions():
    """Far ones (10^7: 64-bit angles), negative ones, offsets, shared and strided ones."""
    g = np.random.default_rng(3)
    x, f = _rand(g, (3, 20, 2, 32), "f32"), cn.rotary_frequencies(32)
    pos = torch.from_numpy(g.integers(-10 ** 7, 10 ** 7, (3, 20)).astype(np.int32)).cuda()
    _check(x, f, "far", positions=pos)
    _check(x, f, "offset", offset=10 ** 7 - 3)
    _check(x, f, "both", positions=pos, offset=-1000)
    _check(x, f, "shared", positions=pos[0])
    _check(x, f, "expanded", positions=pos[:1].expand(3, 20))
    wide = torch.from_numpy(g.integers(0, 9999, (3, 41)).astype(np.int32)).cuda()
    y = cn.rotary(x, f, positions=wide[:, :20])
    assert torch.equal(y, cn.rotary(x, f, positions=wide[:, :20].contiguous()))
    for scaling in ("linear", "ntk", "yarn"):
        s = cn.rotary_frequencies(32, 500000.0, scaling=scaling, factor=8.0, original_length=4096)
        _check(x, s, scaling, positions=pos)


@pytest.mark.parametrize("dt", list(DT))
def test_strides_and_in_place(dt):
    """Heads inside a projection's rows, odd offsets, transposed heads, in place in all of them."""
    g = np.random.default_rng(4)
    f = cn.rotary_frequencies(32)
    rows = _rand(g, (2, 13, 400), dt)
    cuts = {"rows": lambda t: t[..., :320].unflatten(-1, (5, 64)), "odd": lambda t: t[..., 3:323].unflatten(-1, (5, 64)),
            "parts": lambda t: t[..., :384].unflatten(-1, (3, 128))[..., 64:],
            "positions": lambda t: t[:, ::2, 16:336].unflatten(-1, (5, 64)),
            "transposed": lambda t: t[..., :320].reshape(2, 5, 13, 64).transpose(1, 2)}
    for inter in (True, False):
        for name, cut in cuts.items():
            x = cut(rows)
            y = _check(x, f, name, interleaved=inter)
            want = cn.rotary(x, f, interleaved=inter)
            copy = rows.clone()
            part = cut(copy) if name != "transposed" else cut(copy).contiguous().transpose(1, 2).contiguous().transpose(1, 2)
            got = cn.rotary(part, f, interleaved=inter, out=part)
            assert got.data_ptr() == part.data_ptr() and torch.equal(bits(got), bits(want)), name
            if name in ("rows", "odd", "parts", "positions"):  # what lies between stays
                cut(copy).zero_()
                left = rows.clone()
                cut(left).zero_()
                assert torch.equal(bits(copy), bits(left)), name
        shared = _rand(g, (2, 13, 1, 64), dt).expand(2, 13, 4, 64)
        _check(shared, f, "shared", interleaved=inter)


def test_offsets_past_32_bits():
    far = (1 << 31) + 64
    buf = torch.empty(far + 256, dtype=torch.bfloat16, device="cuda")
    x = buf.as_strided((1, 2, 2, 64), (far, far, 64, 1))
    x.copy_(_rand(np.random.default_rng(5), (1, 2, 2, 64), "bf16"))
    _check(x, cn.rotary_frequencies(64), "far")
    want = cn.rotary(x, cn.rotary_frequencies(64))
    cn.rotary(x, cn.rotary_frequencies(64), out=x)
    assert torch.equal(x, want)


def test_as_many_heads_as_there_can_be():
    """Head counts whose steps pass 32 bits; every head the same, in and out."""
    h = (1 << 31) - 1
    row = torch.tensor([0.5, -2.0, 3.0], dtype=torch.bfloat16, device="cuda")
    x = torch.empty(1, 1, h, 3, dtype=row.dtype, device="cuda")
    for part in x[0, 0].split(1 << 28):
        part.copy_(row.expand_as(part))
    y = cn.rotary(x, cn.rotary_frequencies(2), offset=1)
    del x
    one = row.expand(1, 1, 1, 3).contiguous()
    _check(one, cn.rotary_frequencies(2), "one head", offset=1)
    want = cn.rotary(one, cn.rotary_frequencies(2), offset=1)
    assert all(torch.equal(part, want[0, 0].expand_as(part)) for part in y[0, 0].split(1 << 28))


def test_infinity_and_nan_stay_in_their_pairs():
    g = np.random.default_rng(6)
    x, f = _rand(g, (1, 4, 2, 16), "f32"), cn.rotary_frequencies(8)
    clean = cn.rotary(x, f, interleaved=True)
    x[0, 1, 0, 3], x[0, 2, 1, 12] = float("nan"), float("inf")
    y = cn.rotary(x, f, interleaved=True)
    assert torch.isnan(y[0, 1, 0, 2:4]).all() and y[0, 2, 1, 12] == float("inf")
    y[0, 1, 0, 2:4], y[0, 2, 1, 12] = clean[0, 1, 0, 2:4], clean[0, 2, 1, 12]
    assert torch.equal(y, clean)


def test_gradient_against_differences():
    g = np.random.default_rng(7)
    x, dy, f = _rand(g, (2, 5, 2, 12), "f32"), _rand(g, (2, 5, 2, 12), "f32"), cn.rotary_frequencies(10)
    for inter in (True, False):
        dx = R.f64(cn.rotary_backward(dy, f, offset=3, interleaved=inter, scale=1.5))
        num, v = R.directional(lambda x: A.rotary(x, f.cpu(), torch.arange(5) + 3, inter, 1.5)[:1], dict(x=R.f64(x)), "x",
                               (R.f64(dy),))
        assert abs(num - float((dx * v).sum())) <= 1e-6 * float((dx * v).abs().sum())


def test_graph_and_streams():
    g = np.random.default_rng(8)
    x, f = _rand(g, (16, 8, 128), "bf16"), cn.rotary_frequencies(128)
    pos = torch.arange(16, dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        cn.rotary(x, f, positions=pos)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = cn.rotary(x, f, positions=pos)
    for i in range(3):
        pos += 7
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, cn.rotary(x, f, positions=pos)), i


def test_empty_and_refusals():
    f = cn.rotary_frequencies(16)
    assert cn.rotary(torch.zeros(2, 0, 3, 16, device="cuda"), f).shape == (2, 0, 3, 16)
    x = torch.zeros(2, 4, 3, 16, device="cuda")
    pos = torch.zeros(2, 4, dtype=torch.int32, device="cuda")
    for bad, kind in ((lambda: cn.rotary(x.cpu(), f), TypeError), (lambda: cn.rotary(x.double(), f), TypeError),
                      (lambda: cn.rotary(x[0, 0], f), ValueError), (lambda: cn.rotary(x, f.float()), TypeError),
                      (lambda: cn.rotary(x, f.cpu()), TypeError), (lambda: cn.rotary(x[..., :8], f), ValueError),
                      (lambda: cn.rotary(x.transpose(2, 3), cn.rotary_frequencies(2)), ValueError),
                      (lambda: cn.rotary(x, f, positions=pos.long()), TypeError),
                      (lambda: cn.rotary(x, f, positions=pos[:, :3]), ValueError),
                      (lambda: cn.rotary(x[:, 0], f, positions=pos), ValueError),
                      (lambda: cn.rotary(x, f, offset=1 << 50), cn.CnhwcError),
                      (lambda: cn.rotary(x, f, out=x[:, :, :1].expand(x.shape)), cn.CnhwcError),
                      (lambda: cn.rotary(x, f, out=x.half()), TypeError),
                      (lambda: cn.rotary(x[:1].expand(x.shape), f, out=x), cn.CnhwcError)):
        with pytest.raises(kind):
            bad()
