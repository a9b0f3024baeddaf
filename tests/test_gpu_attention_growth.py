"""Linear attention's states under decays that leave fp32's ordinary range: infinite states."""
import numpy as np
import pytest
import torch

import seq_reference as R

pytestmark = pytest.mark.gpu

cn = pytest.importorskip("convolution_nhwc_conv2d_amd")

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def _rows(seed, dt, n, l, h, dk, dv):
    g = np.random.default_rng(seed)
    r = lambda *sh: R.rand(g, *sh).to(DT[dt]).cuda()
    return r(n, l, h, dk), r(n, l, h, dk), r(n, l, h, dv), r(n, l, h, dv)


@pytest.mark.parametrize("dt", list(DT))
def test_an_infinite_state_stays_infinite(dt):
    """Through a token and through the runs of a prompt alike, and only where it is: each decay
    (of a token, of a chunk and of a run) is e^-0.5 or faster and no underflow."""
    q, k, v, _ = _rows([1], dt, 1, 700, 2, 64, 64)
    state = torch.zeros(1, 2, 64, 64, device="cuda")
    state[0, 1, 3, 5], state[0, 0, 60, 63] = float("inf"), float("-inf")
    hit = torch.isinf(state)
    was = state.clone()
    cn.linear_attention_step(q[:, 0], k[:, 0], v[:, 0], torch.tensor([-0.5, -1.0], device="cuda"), state)
    assert torch.equal(state[hit], was[hit]) and torch.isfinite(state[~hit]).all()
    assert cn.linear_attention_workspace_bytes(q, v) > 0  # more than one run
    _, last = cn.linear_attention(q, k, v, torch.tensor([-0.02, -0.05], device="cuda"), state=was, return_state=True)
    assert torch.equal(last[hit], was[hit]) and torch.isfinite(last[~hit]).all()
