"""The example block: prompts and tokens agree, its gradient is the one that
differences of its own forward pass give, and it learns."""
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


def test_tokens_follow_ragged_prompts(ex):
    """In float32 the paths differ by the order of the projections' sums alone:
    a few hundred terms, 2^-24 each, through two projections and the scan."""
    block = ex.SequenceBlock(64, 96, dtype=torch.float32)
    lengths = torch.tensor([40, 1, 17, 0], dtype=torch.int32, device="cuda")
    x = torch.randn(4, 40, 64, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    tok = torch.randn(4, 5, 64, generator=torch.Generator(device="cuda").manual_seed(2), device="cuda")
    y, by_token = ex.answer(block, x, lengths, tok)
    for n, m in enumerate([40, 1, 17, 0]):
        whole, _ = block.forward(torch.cat([x[n, :m], tok[n]], 0)[None].contiguous())
        scale = float(whole.abs().max())
        assert float((whole[0, :m] - y[n, :m]).abs().max() if m else 0.0) < 2e-5 * scale
        assert float((whole[0, m:] - by_token[n]).abs().max()) < 2e-5 * scale


def test_gradient_against_differences(ex):
    """Directional differences of the float32 block with a step of 2^-7: the error
    is the third derivative times 2^-14 / 6 and the rounding of the loss, 2^-24
    of its magnitude over 2^-7; both stay below 1% of the gradients' scale."""
    block = ex.SequenceBlock(32, 48, states=8, rank=8, dtype=torch.float32)
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(2, 24, 32, generator=g, device="cuda")
    w = torch.randn(2, 24, 32, generator=g, device="cuda")
    lengths = torch.tensor([24, 9], dtype=torch.int32, device="cuda")
    keep = {}
    block.forward(x, lengths=lengths, keep=keep)
    dx, grads = block.backward(w, keep)

    def loss(xx):
        return float((block.forward(xx, lengths=lengths)[0].double() * w.double()).sum())
    step = 2.0 ** -7
    for name, grad in [("x", dx)] + sorted(grads.items()):
        v = grad / grad.norm()  # along the gradient: the derivative is its norm
        if name == "x":
            num = (loss(x + step * v) - loss(x - step * v)) / (2 * step)
        else:
            t = block.p[name]
            old = t.clone()
            t.copy_(old + step * v)
            up = loss(x)
            t.copy_(old - step * v)
            num = (up - loss(x)) / (2 * step)
            t.copy_(old)
        assert abs(num - float(grad.norm())) < 1e-2 * float(grad.norm()), name


def test_it_learns(ex):
    losses = ex.train(ex.SequenceBlock(32, 64, dtype=torch.float32), steps=40)
    assert losses[-1] < 0.8 * losses[0]
