"""Sequence operators over very many sequences."""
import pytest
import torch

pytestmark = pytest.mark.gpu

cn = pytest.importorskip("convolution_nhwc_conv2d_amd")


@pytest.mark.parametrize("c", [2, 3])
def test_conv_gradient_of_sixteen_million_sequences(c):
    """2^24 sequences of one position, each with a workgroup of its own: more than
    one launch takes.  Small whole numbers without activation, so every sum is
    exact in 32 bits in any order."""
    n, k = 1 << 24, 4
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randint(-1, 2, (n, 1, c), generator=g, device="cuda").float()
    dy = torch.randint(-1, 2, (n, 1, c), generator=g, device="cuda").float()
    w = torch.randint(-3, 4, (c, k), generator=g, device="cuda").float()
    r = cn.causal_conv1d_backward(dy, x, w, torch.zeros(c, device="cuda"))
    assert torch.equal(r.x, dy * w[:, k - 1])
    assert torch.equal(r.bias, dy.sum((0, 1), dtype=torch.float64).float())
    assert not r.w[:, :k - 1].any()
    assert torch.equal(r.w[:, k - 1], (dy * x).sum((0, 1), dtype=torch.float64).float())
