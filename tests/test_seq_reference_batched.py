"""The batched 64-bit references against the step-by-step ones (CPU only)."""
import numpy as np
import pytest
import torch

import seq_reference as R
import seq_reference_batched as B


def _same(got, want):
    assert got.shape == want.shape and torch.allclose(got, want, rtol=1e-12, atol=1e-13)


@pytest.mark.parametrize("lengths", [None, [9, 0, 1, 5], [12, -2, 9, 3]])
@pytest.mark.parametrize("act", [False, True])
@pytest.mark.parametrize("k", [1, 3, 8])
def test_causal_conv(k, act, lengths):
    g = np.random.default_rng(k)
    n, l, c = 4, 9, 3
    x, dy = R.rand(g, n, l, c).double(), R.rand(g, n, l, c).double()
    w, b = R.rand(g, c, k).double(), R.rand(g, c).double()
    lengths = None if lengths is None else torch.tensor(lengths, dtype=torch.int32)
    for state, bias, dlast in ((None, None, None), (R.rand(g, n, k - 1, c).double(), b, R.rand(g, n, k - 1, c).double())):
        for got, want in zip(B.causal_conv(x, w, bias, act, state, lengths), R.causal_conv(x, w, bias, act, state, lengths)):
            _same(got, want)
        for absolute in (False, True):
            args = (dy, x, w, bias, act, state, lengths, dlast)
            for got, want in zip(B.causal_conv_backward(*args, absolute=absolute), R.causal_conv_backward(*args, absolute=absolute)):
                _same(got, want)


@pytest.mark.parametrize("lengths", [None, [7, 0, 3], [9, -1, 7]])
@pytest.mark.parametrize("plus", [False, True])
def test_scan(plus, lengths):
    g = np.random.default_rng(5)
    n, l, d, s = 3, 7, 4, 5
    r = lambda *sh, **kw: R.rand(g, *sh, **kw).double()
    lengths = None if lengths is None else torch.tensor(lengths, dtype=torch.int32)
    whole = [r(n, l, d), r(n, l, d, scale=0.5).abs(), -r(d, s).abs(), r(n, l, s), r(n, l, s)]
    for rest in ([None, None, None, plus, None, lengths],
                 [r(d), r(n, l, d), r(d).abs() * 0.2, plus, r(n, d, s), lengths]):
        dlast = None if rest[0] is None else r(n, d, s)
        for absolute in (False, True):
            args = whole + rest
            for got, want in zip(B.scan(*args, absolute=absolute), R.scan(*args, absolute=absolute)):
                _same(got, want)
            dy = r(n, l, d)
            got = B.scan_backward(dy, *args, dlast, absolute=absolute)
            want = R.scan_backward(dy, *args, dlast, absolute=absolute)
            for name in want:
                if name == "gate" and rest[1] is None or name == "skip" and rest[0] is None:
                    continue
                _same(got[name], want[name])
