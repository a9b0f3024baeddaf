"""Every component of the example block's gradient against automatic
differentiation of the block in 64 bits.

The bound: the stages of the block add up at most 32 L + 128 = 896 roundings in
the scan, 256 in the norm, 64 in the convolution and 100 in each of four
projections, forward and back: below 4000 of 2^-24, 2.4e-4 of the terms.  Sums
of a few hundred terms of random sign are a tenth of their magnitudes or more at
the largest component, which the difference is compared with: 2.4e-3.
"""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

cn = pytest.importorskip("convolution_nhwc_conv2d_amd")
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "sequence_block.py")


@pytest.fixture(scope="module")
def ex():
    spec = importlib.util.spec_from_file_location("sequence_block", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _model(p, x, lengths, inner, states, taps):
    """The block by its formulas, each sequence cut to its own length."""
    silu = lambda t: t / (1 + torch.exp(-t))
    out = []
    for i, m in enumerate(lengths):
        xi = x[i, :m]
        xc = xi - xi.mean(-1, keepdim=True)
        h = xc / torch.sqrt(xc.square().mean(-1, keepdim=True) + 1e-5) * p["norm_w"] + p["norm_b"]
        v, z = (h @ p["w_in"].t()).split(inner, -1)
        rows = torch.cat([torch.zeros(taps - 1, inner, dtype=x.dtype), v], 0)
        u = silu(p["conv_b"] + sum(rows[j:j + m] * p["conv_w"][:, j] for j in range(taps)))
        step = torch.log1p(torch.exp(u @ p["w_rank"].t() @ p["w_delta"].t() + p["delta_bias"]))
        b, c = (u @ p["w_bc"].t()).split(states, -1)
        a, s, ys = -torch.exp(p["a_log"]), torch.zeros(inner, states, dtype=x.dtype), []
        for t in range(m):
            s = torch.exp(step[t][:, None] * a) * s + (step[t] * u[t])[:, None] * b[t]
            ys.append((s * c[t]).sum(-1) + p["skip"] * u[t])
        out.append(xi + (torch.stack(ys) * silu(z)) @ p["w_out"].t())
    return out


@pytest.mark.parametrize("lengths", [[24, 24], [24, 9]])
def test_gradient_component_by_component(ex, lengths):
    block = ex.SequenceBlock(32, 48, states=8, rank=8, dtype=torch.float32)
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn(2, 24, 32, generator=g, device="cuda")
    w = torch.randn(2, 24, 32, generator=g, device="cuda")
    keep = {}
    y, _ = block.forward(x, lengths=torch.tensor(lengths, dtype=torch.int32, device="cuda"), keep=keep)
    dx, grads = block.backward(w, keep)
    p = {k: v.detach().cpu().double().requires_grad_() for k, v in block.p.items()}
    xd = x.cpu().double().requires_grad_()
    out = _model(p, xd, lengths, 48, 8, 4)
    loss = sum((o * w[i, :len(o)].cpu().double()).sum() for i, o in enumerate(out))
    names = sorted(p)
    want = dict(zip(["x"] + names, torch.autograd.grad(loss, [xd] + [p[k] for k in names])))
    for i, m in enumerate(lengths):  # past a length the block passes x on, and its gradient
        scale = float(out[i].detach().abs().max())
        assert float((y[i, :m].cpu().double() - out[i].detach()).abs().max()) <= 2.4e-3 * scale
        want["x"][i, m:] += w[i, m:].cpu().double()
    assert set(grads) == set(names)
    for name, t in [("x", dx)] + sorted(grads.items()):
        ref = want[name]
        assert t.shape == ref.shape and float(ref.abs().max()) > 0, name
        assert float((t.cpu().double() - ref).abs().max()) <= 2.4e-3 * float(ref.abs().max()), name
