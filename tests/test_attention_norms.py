"""The norm's bound of linear attention notices mistakes planted in the reference (on the CPU)."""
import numpy as np
import pytest
import torch

import attention_norms as N
import attention_reference as A
import seq_reference as R


def _inputs(l, life, big):
    g = np.random.default_rng([1, l])
    r = lambda *sh: R.rand(g, *sh).double()
    decay = torch.tensor([-np.log(2.0) / life], dtype=torch.float64)
    return r(1, l, 1, 32), r(1, l, 1, 32), r(1, l, 1, 24), decay, r(1, 1, 32, 24) * big


def _apart(l, life, big, change):
    """How far y is with `change` in the carried state's place at every 32nd position."""
    q, k, v, g, s0 = _inputs(l, life, big)
    want, _ = A.attention(q, k, v, g, 1.0, s0, None)
    parts, s = [], s0
    for t in range(0, l, 32):
        y, s = A.attention(q[:, t:t + 32], k[:, t:t + 32], v[:, t:t + 32], g, 1.0, s, None)
        parts.append(y)
        s = change(s)
    return N.far(torch.cat(parts, 1), want, (1, 3))


BOUND = N.BOUND[torch.bfloat16]  # the widest


@pytest.mark.parametrize("life", [40, 4096])
def test_what_the_bound_notices(life):
    """A carried state that is 5% off once, or always by what a decay of one position makes;
    one that is lost, or has lost a column's half."""
    once = iter([1.05] + [1.0] * 100)
    assert _apart(96, 4096, 30, lambda s: s * next(once)) > BOUND
    assert _apart(640, life, 1, lambda s: s * 0.0) > 10 * BOUND
    assert _apart(640, life, 1, lambda s: torch.cat([s[:, :, :16], s[:, :, 16:] * 0], 2)) > 10 * BOUND
    assert _apart(640, life, 1, lambda s: s * 0.95) > BOUND
    q, k, v, g, s0 = _inputs(640, life, 1)
    want, _ = A.attention(q, k, v, g, 1.0, s0, None)
    # products in 3 bits: those of q and k rounded to an eighth of themselves
    rough = lambda t: torch.ldexp(torch.round(torch.frexp(t)[0] * 8) / 8, torch.frexp(t)[1])
    assert N.far(A.attention(rough(q), k, v, g, 1.0, s0, None)[0], want, (1, 3)) > BOUND
    assert N.far(want * 0, want, (1, 3)) > BOUND


def test_what_it_lets_pass():
    """The 64-bit values with q, k, v and y rounded to bf16 once each are within half of it."""
    q, k, v, g, s0 = _inputs(640, 40, 1)
    want, _ = A.attention(q, k, v, g, 1.0, s0, None)
    near = lambda t: t.bfloat16().double()
    y = near(A.attention(near(q), k, v, g, 1.0, near(s0), None)[0])
    assert N.far(y, want, (1, 3)) < BOUND / 2
    N.check(want.float(), want, (1, 3), "rounded to fp32")
    with pytest.raises(AssertionError):
        N.check((want * 1.01).bfloat16(), want, (1, 3), "1% off")


def test_every_argument_by_its_absolute_value():
    """The magnitudes of the bounds are those of the same formula on absolute values."""
    q, k, v, g, s0 = _inputs(40, 40, 1)
    y, s = A.attention(q, k, v, g, 1.0, s0, None)
    q, k, v, s0 = A.absolute(q, k, v, s0)
    my, ms = A.attention(q, k, v, g, 1.0, s0, None)
    assert bool((my >= y.abs()).all()) and bool((ms >= s.abs()).all())
