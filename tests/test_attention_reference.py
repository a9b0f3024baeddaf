"""The 64-bit references of the root-mean-square norm, rotary positions and linear
attention against other forms of the same definitions (no GPU): automatic
differentiation, complex numbers, the product of all positions with all
positions, differences, and a planted mistake that they must notice."""
import math

import pytest
import torch

import attention_reference as A
import convolution_nhwc_conv2d_amd as cn


def _rand(*shape, seed=0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed), dtype=torch.float64)


@pytest.mark.parametrize("dsum", [True, False])
def test_rms_norm_gradient(dsum):
    x, w, dy = _rand(5, 12), _rand(12, seed=1), _rand(5, 12, seed=2)
    more = _rand(5, 12, seed=3) if dsum else None
    x.requires_grad_(), w.requires_grad_()
    y, z, rstd, _ = A.rms_norm(x, None, w, 1e-6)
    loss = (y * dy).sum() + (0 if more is None else (z * more).sum())
    want = torch.autograd.grad(loss, (x, w))
    got = A.rms_norm_backward(dy, x.detach(), rstd.detach(), w.detach(), more)
    for a, b in zip(got, want):
        assert torch.allclose(a, b, rtol=1e-12, atol=1e-12)
    y2 = torch.nn.functional.rms_norm(x.detach(), (12,), w.detach(), 1e-6)
    assert torch.allclose(y.detach(), y2, rtol=1e-12, atol=1e-12)


@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("r", [0, 6, 10])
def test_rotary_is_a_turn(interleaved, r):
    x, f = _rand(2, 7, 3, 10), cn.rotary_frequencies(r, device="cpu")
    at = torch.arange(7) + torch.tensor([[0], [100000]])
    y, _ = A.rotary(x, f, at, interleaved, 1.5)
    part = x[..., :r].unflatten(-1, (r // 2, 2) if interleaved else (2, r // 2))
    axis = -1 if interleaved else -2
    z = torch.complex(*part.unbind(axis)) * torch.polar(torch.tensor(1.5, dtype=torch.float64),
                                                        at.double()[..., None, None] * f)
    z = torch.stack([z.real, z.imag], axis).flatten(-2)
    assert torch.allclose(y, torch.cat([z, x[..., r:]], -1), rtol=1e-9, atol=1e-9)
    back, _ = A.rotary(y, f, at, interleaved, 1 / 1.5, -1)
    assert torch.allclose(back, x, rtol=1e-12, atol=1e-12)
    if r:  # a turn the wrong way is noticed
        wrong, _ = A.rotary(x, f, at, interleaved, 1.5, -1)
        assert not torch.allclose(wrong, y, atol=1e-3)


def test_frequencies():
    f = cn.rotary_frequencies(64, 10000.0, device="cpu")
    assert f.dtype == torch.float64 and f.shape == (32,)
    for i in (0, 1, 17, 31):
        assert abs(float(f[i]) - 10000.0 ** (-2 * i / 64)) < 1e-15
    assert torch.allclose(cn.rotary_frequencies(64, scaling="linear", factor=4.0, device="cpu"), f / 4)
    ntk = cn.rotary_frequencies(64, scaling="ntk", factor=8.0, device="cpu")
    assert float(ntk[0]) == 1.0 and abs(float(ntk[-1] / f[-1]) - 1 / 8) < 1e-12
    yarn = cn.rotary_frequencies(64, scaling="yarn", factor=16.0, original_length=2048, device="cpu")
    turns = f * 2048 / (2 * math.pi)
    assert torch.equal(yarn[turns > 32], f[turns > 32]) and (turns > 32).any()
    assert torch.allclose(yarn[turns < 1], f[turns < 1] / 16, rtol=1e-14) and (turns < 1).any()
    assert ((yarn <= f) & (yarn >= f / 16 * (1 - 1e-14))).all()
    assert cn.rotary_frequencies(0, device="cpu").shape == (0,)
    for bad in (dict(dim=3), dict(dim=-2), dict(dim=4, scaling="other"), dict(dim=4, base=0.0),
                dict(dim=4, factor=-1.0), dict(dim=4, scaling="yarn"),
                dict(dim=4, scaling="yarn", original_length=8, fast=1.0, slow=2.0)):
        with pytest.raises(ValueError):
            cn.rotary_frequencies(device="cpu", **bad)


def _attention(seed=0, n=3, l=9, h=2, dk=4, dv=5):
    return dict(q=_rand(n, l, h, dk, seed=seed), k=_rand(n, l, h, dk, seed=seed + 1), v=_rand(n, l, h, dv, seed=seed + 2),
                g=-_rand(h, seed=seed + 3).abs(), scale=0.7, state=_rand(n, h, dk, dv, seed=seed + 4))


def _all_pairs(q, k, v, g, scale, state, lengths):
    """The product of all positions with all positions."""
    n, l = q.shape[:2]
    t = torch.arange(l)
    far = (t[:, None] - t).double()
    between = torch.where(far >= 0, torch.exp(g[:, None, None] * far.clamp(min=0)), 0.0)
    m = torch.full((n,), l) if lengths is None else lengths
    live = (t < m[:, None]).double()
    p = torch.einsum("nuhd,nshd->nhus", q, k) * between
    before = torch.exp(g[:, None] * (t + 1.0))
    y = torch.einsum("nhus,nshe->nuhe", p, v) + torch.einsum("hu,nuhd,nhde->nuhe", before, q, state)
    ahead = (m[:, None] - 1 - t).double()
    w = torch.where(ahead >= 0, 1.0, 0.0)[:, None] * torch.exp(g[:, None] * ahead.clamp(min=0)[:, None])
    s = torch.einsum("nhs,nshd,nshe->nhde", w, k, v) + torch.exp(g * m[:, None])[..., None, None] * state
    return scale * y * live[:, :, None, None], s


@pytest.mark.parametrize("lengths", [None, [9, 0, 4]])
def test_attention_against_all_pairs_and_its_gradient(lengths):
    a = _attention()
    lengths = None if lengths is None else torch.tensor(lengths)
    y, s = A.attention(**a, lengths=lengths)
    leaves = {k: a[k].clone().requires_grad_() for k in ("q", "k", "v", "g", "state")}
    y2, s2 = _all_pairs(**{**a, **leaves}, lengths=lengths)
    assert torch.allclose(y, y2.detach(), rtol=1e-12, atol=1e-12)
    assert torch.allclose(s, s2.detach(), rtol=1e-12, atol=1e-12)
    dy, ds = _rand(*y.shape, seed=7), _rand(*s.shape, seed=8)
    want = torch.autograd.grad((y2 * dy).sum() + (s2 * ds).sum(), list(leaves.values()))
    got = A.attention_backward(dy, **a, lengths=lengths, dlast=ds)
    for name, w in zip(("q", "k", "v", "log_decay", "state"), want):
        assert torch.allclose(got[name], w, rtol=1e-11, atol=1e-11), name
    wrong = A.attention_backward(dy, **{**a, "g": a["g"] * 1.01}, lengths=lengths, dlast=ds)
    assert not any(torch.allclose(wrong[n], got[n], rtol=1e-6) for n in ("q", "k", "v", "log_decay", "state"))
