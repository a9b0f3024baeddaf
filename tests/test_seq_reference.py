"""The 64-bit references of the sequence operators against closed forms, library
operations, automatic differentiation and central differences (CPU only), and a
planted mistake that these have to find."""
import numpy as np
import pytest
import torch

import seq_reference as R


def _scan_inputs(n=2, l=7, d=3, s=4, seed=1):
    g = np.random.default_rng(seed)
    r = lambda *sh, **kw: R.rand(g, *sh, **kw).double()
    return dict(u=r(n, l, d), delta=r(n, l, d, scale=0.5), a=-r(d, s).abs() - 0.2, b=r(n, l, s), c=r(n, l, s),
                skip=r(d), gate=r(n, l, d), bias=r(d), state=r(n, d, s))


def _scan(u, delta, a, b, c, skip, gate, bias, state, lengths=None):
    return R.scan(u, delta, a, b, c, skip, gate, bias, True, state, lengths)


def test_layer_norm_is_the_library_one():
    g = np.random.default_rng(0)
    x, w, b = R.rand(g, 5, 9).double(), R.rand(g, 9).double(), R.rand(g, 9).double()
    y, mean, rstd, _ = R.layer_norm(x, w, b, 1e-5)
    assert torch.allclose(y, torch.nn.functional.layer_norm(x, (9,), w, b, 1e-5), rtol=1e-13, atol=1e-13)
    dy = R.rand(g, 5, 9).double()
    leaves = [t.clone().requires_grad_() for t in (x, w, b)]
    want = torch.autograd.grad(torch.nn.functional.layer_norm(leaves[0], (9,), leaves[1], leaves[2], 1e-5), leaves, dy)
    for a, e in zip(R.layer_norm_backward(dy, x, mean, rstd, w), want):
        assert torch.allclose(a, e, rtol=1e-11, atol=1e-12)


@pytest.mark.parametrize("k", [1, 2, 4])
def test_causal_conv_is_a_padded_grouped_conv(k):
    g = np.random.default_rng(k)
    x, w, b = R.rand(g, 2, 6, 3).double(), R.rand(g, 3, k).double(), R.rand(g, 3).double()
    y, last, _ = R.causal_conv(x, w, b, False, None, None)
    lib = torch.nn.functional.conv1d(torch.nn.functional.pad(x.transpose(1, 2), (k - 1, 0)), w[:, None], b, groups=3)
    assert torch.allclose(y, lib.transpose(1, 2), rtol=1e-13, atol=1e-13)
    assert torch.equal(last, x[:, 6 - (k - 1):])


def test_causal_conv_gradient():
    g = np.random.default_rng(3)
    lengths = torch.tensor([6, 0, 2], dtype=torch.int32)
    ins = dict(x=R.rand(g, 3, 6, 2).double(), w=R.rand(g, 2, 4).double(), b=R.rand(g, 2).double(),
               state=R.rand(g, 3, 3, 2).double())
    dy, dl = R.rand(g, 3, 6, 2).double(), R.rand(g, 3, 3, 2).double()
    got = dict(zip(("x", "w", "b", "state"), R.causal_conv_backward(dy, ins["x"], ins["w"], ins["b"], True,
                                                                     ins["state"], lengths, dl)))
    f = lambda x, w, b, state: R.causal_conv(x, w, b, True, state, lengths)[:2]
    for name in ins:
        num, v = R.directional(f, ins, name, (dy, dl))
        assert abs(num - float((got[name] * v).sum())) < 1e-7 * (1 + abs(num)), name


def test_scan_of_one_state_is_a_geometric_sum():
    """Constant decay: h[t] = sum_k r^k, y = c h."""
    l = 5
    one = torch.ones(1, l, 1, dtype=torch.float64)
    a = torch.full((1, 1), -0.3, dtype=torch.float64)
    y, last = R.scan(one, one, a, one, 2 * one, None, None, None, False, None, None)
    r = float(np.exp(-0.3))
    want = [2 * (1 - r ** (t + 1)) / (1 - r) for t in range(l)]
    assert np.allclose(y[0, :, 0].numpy(), want, rtol=1e-13)
    assert np.allclose(last.item(), want[-1] / 2, rtol=1e-13)


def test_scan_state_hand_over_and_lengths():
    ins = _scan_inputs()
    y, last = _scan(**ins)
    seq = ("u", "delta", "b", "c", "gate")
    first = {k: (v[:, :3] if k in seq else v) for k, v in ins.items()}
    rest = {k: (v[:, 3:] if k in seq else v) for k, v in ins.items()}
    y1, s1 = _scan(**first)
    y2, s2 = _scan(**{**rest, "state": s1})
    assert torch.allclose(torch.cat([y1, y2], 1), y, rtol=1e-14) and torch.allclose(s2, last, rtol=1e-14)
    yl, sl = _scan(**ins, lengths=torch.tensor([3, 0]))
    assert torch.equal(yl[0, :3], y1[0]) and torch.equal(sl[0], s1[0]) and torch.equal(sl[1], ins["state"][1])
    assert not yl[0, 3:].any() and not yl[1].any()


@pytest.mark.parametrize("lengths", [None, [7, 0], [1, 5]])
def test_scan_gradient(lengths):
    ins = _scan_inputs()
    lengths = None if lengths is None else torch.tensor(lengths, dtype=torch.int32)
    g = np.random.default_rng(9)
    dy, dl = R.rand(g, 2, 7, 3).double(), R.rand(g, 2, 3, 4).double()
    got = R.scan_backward(dy, ins["u"], ins["delta"], ins["a"], ins["b"], ins["c"], ins["skip"], ins["gate"],
                          ins["bias"], True, ins["state"], lengths, dl)
    f = lambda **kw: _scan(**kw, lengths=lengths)
    for name in ins:
        num, v = R.directional(f, ins, name, (dy, dl))
        assert abs(num - float((got[name] * v).sum())) < 2e-7 * (1 + abs(num)), name


def test_a_planted_mistake_is_found():
    """A gradient that forgets one decay does not match the differences."""
    ins = _scan_inputs()
    dy = R.rand(np.random.default_rng(9), 2, 7, 3).double()
    wrong = dict(ins, a=ins["a"] * 0.9)
    got = R.scan_backward(dy, wrong["u"], wrong["delta"], wrong["a"], wrong["b"], wrong["c"], wrong["skip"],
                          wrong["gate"], wrong["bias"], True, wrong["state"], None, None)
    num, v = R.directional(lambda **kw: _scan(**kw), ins, "u", (dy, None))
    assert abs(num - float((got["u"] * v).sum())) > 1e-4 * abs(num)
