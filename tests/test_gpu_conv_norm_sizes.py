"""The causal convolution and layer norm at sizes whose loops small ones do not
run, against 64-bit references on the GPU.

The convolution gives a thread more than four positions from 655360 vectors on
(of 16 bytes, or single elements; 32 positions at most), its gradient from
983040 pairs or single elements, 1966080 in batches with lengths (64 rows at
most).  Layer norm goes round its row loop again beyond 8192 workgroups.  Bounds as for the small sizes.
"""
import pytest
import torch

import seq_reference as R
import seq_reference_batched as B

pytestmark = pytest.mark.gpu

cn = pytest.importorskip("convolution_nhwc_conv2d_amd")

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def _check(got, ref, mag, k, where):
    R.check(got, ref.cpu(), mag.cpu(), k, where)


def _conv(seed, n, l, c, k, dt, lengths, wide):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *sh, scale=1.0: (torch.randn(sh, generator=g, device="cuda") * scale).to(DT[dt])
    x = r(n, l, 2 * c)[..., :c] if wide else r(n, l, c)
    return dict(x=x, w=r(c, k, scale=k ** -0.5), b=r(c, scale=0.3), state=r(n, k - 1, c), dy=r(n, l, c), dstate=r(n, k - 1, c),
                lengths=None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda"))


CONV = [  # runs of 8, 12, 16 and 32 positions; vectors, strided vectors and single elements
    ("f32", 3, 3501, 256, 4, [3501, 0, 3499], False), ("bf16", 3, 4001, 1024, 4, None, True),
    ("f16", 3, 2005, 301, 3, [2005, 1, 1997], False), ("bf16", 4, 8200, 1024, 4, [8200, 8199, 33, 4097], False),
    ("f32", 2, 8195, 267, 8, None, True), ("f16", 2, 4103, 1024, 2, [4100, 3], False),
]


@pytest.mark.parametrize("dt,n,l,c,k,lengths,wide", CONV, ids=lambda v: "ragged" if isinstance(v, list) else str(v))
def test_conv_forward(dt, n, l, c, k, lengths, wide):
    i = _conv(1, n, l, c, k, dt, lengths, wide)
    y, last = cn.causal_conv1d(i["x"], i["w"], i["b"], activation="silu", state=i["state"], lengths=i["lengths"],
                               return_state=True)
    ry, rl, mag = B.causal_conv(*(i[j].double() for j in ("x", "w", "b")), True, i["state"].double(), i["lengths"])
    _check(y, ry, mag, 32, "y")
    assert torch.equal(last.double(), rl)


GRAD = [  # runs of 4 to 64 rows; pairs, strided pairs and single elements
    ("f32", 3, 4200, 512, 4, [4200, 0, 4197], False), ("f16", 2, 4203, 512, 4, [17, 4201], True),
    ("f32", 3, 4200, 256, 4, [4200, 0, 4197], False), ("f32", 2, 7001, 384, 3, None, True),
    ("f16", 3, 4011, 300, 7, [4011, 2, 4001], False), ("bf16", 4, 8300, 1024, 4, None, True),
    ("bf16", 6, 8300, 1024, 4, [8300, 8299, 64, 65, 1, 7777], False), ("f32", 3, 8204, 511, 4, [8200, 127, 8204], False),
]


@pytest.mark.parametrize("dt,n,l,c,k,lengths,wide", GRAD, ids=lambda v: "ragged" if isinstance(v, list) else str(v))
def test_conv_backward(dt, n, l, c, k, lengths, wide):
    i = _conv(2, n, l, c, k, dt, lengths, wide)
    r = cn.causal_conv1d_backward(i["dy"], i["x"], i["w"], i["b"], activation="silu", state=i["state"], lengths=i["lengths"],
                                  dstate=i["dstate"])
    args = [i[j].double() for j in ("dy", "x", "w", "b")] + [True, i["state"].double(), i["lengths"], i["dstate"].double()]
    want, mag = B.causal_conv_backward(*args), B.causal_conv_backward(*args, absolute=True)
    many = 64 + n * l
    for name, got, w, m, k_ in zip(("dx", "dw", "dbias", "dstate"), r, want, mag, (64, many, many, 64)):
        _check(got, w, m, k_, name)


@pytest.mark.parametrize("dt,rows,c", [("f32", 8277, 1032), ("f16", 8300, 2051), ("f32", 140001, 64), ("bf16", 33001, 512),
                                       ("bf16", 8500, 4096), ("f16", 66003, 136)])
def test_norm(dt, rows, c):
    g = torch.Generator(device="cuda").manual_seed(3)
    r = lambda *sh, scale=1.0, shift=0.0: (torch.randn(sh, generator=g, device="cuda") * scale + shift).to(DT[dt])
    x, w, b, dy = r(rows, c, scale=1.5, shift=0.5), r(c, scale=0.2, shift=1.0), r(c, scale=0.2), r(rows, c)
    y, mean, rstd = cn.layer_norm(x, w, b, 1e-5, return_stats=True)
    d = [t.double() for t in (x, w, b)]
    ry, rm, rr, mag = R.layer_norm(*d, 1e-5)
    k = 256
    _check(y, ry, mag, k, "y")
    _check(mean, rm, d[0].abs().mean(-1), k, "mean")
    _check(rstd, rr, rr * (1 + d[0].square().mean(-1) * rr * rr), k, "rstd")
    args = [t.double() for t in (dy, x, mean, rstd, w)]
    want, mag = R.layer_norm_backward(*args), R.layer_norm_backward(*args, absolute=True)
    for name, got, v, m, k_ in zip(("dx", "dw", "db"), cn.layer_norm_backward(dy, x, mean, rstd, w), want, mag,
                                   (k, k + rows, k + rows)):
        _check(got, v, m, k_, name)
