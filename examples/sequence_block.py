#!/usr/bin/env python3
"""A residual sequence block out of the package's operators, in the three ways it
is used: prompts of several lengths at once, one token at a time, and training.

    h = layer_norm(x)
    v, z = pointwise conv1d(h)                 halves of one projection's rows
    u = silu(causal_conv1d(v))                 depthwise, K taps
    delta, b, c = pointwise conv1d(u)          what makes the scan selective
    y = selective_scan(u, delta, a, b, c) gated by z
    x + pointwise conv1d(y)

Every product is a conv1d of the package with one tap, the gradients of the
projections too; nothing is recorded for autograd, ``backward`` calls the
operators' backward functions with what ``forward`` kept.

Run it: python examples/sequence_block.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import convolution_nhwc_conv2d_amd as cn  # noqa: E402


def project(x, w):
    """Rows of x [N,L,C] times w [O,C]."""
    return cn.conv1d(x, w[:, None, :])


def project_backward(dy, x, w):
    """dx = dy w, dw = dy^T x: both as one-tap convolutions."""
    dx = project(dy, w.t().contiguous())
    rows = lambda t: t.reshape(-1, t.shape[-1]).t().contiguous()
    return dx, project(rows(x)[None], rows(dy))[0].t().contiguous()


class SequenceBlock:
    """Parameters in `dtype`; a, skip and delta_bias in float32, as the scan takes them."""

    def __init__(self, channels, inner, states=16, taps=4, rank=16, dtype=torch.bfloat16, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)

        def normal(*shape, scale):
            return (torch.randn(shape, generator=g, device=device) * scale).to(dtype)
        step = torch.exp(torch.rand(inner, generator=g, device=device) * 4.6 - 6.9)  # 0.001 to 0.1
        self.p = {
            "norm_w": torch.ones(channels, dtype=dtype, device=device),
            "norm_b": torch.zeros(channels, dtype=dtype, device=device),
            "w_in": normal(2 * inner, channels, scale=channels ** -0.5),
            "conv_w": normal(inner, taps, scale=taps ** -0.5),
            "conv_b": torch.zeros(inner, dtype=dtype, device=device),
            "w_rank": normal(rank, inner, scale=inner ** -0.5),
            "w_delta": normal(inner, rank, scale=rank ** -0.5),
            "w_bc": normal(2 * states, inner, scale=inner ** -0.5),
            "a_log": torch.arange(1, states + 1, device=device).float().log().repeat(inner, 1),
            "skip": torch.ones(inner, device=device),
            "delta_bias": step + torch.log(-torch.expm1(-step)),
            "w_out": normal(channels, inner, scale=inner ** -0.5),
        }
        self.inner, self.states, self.taps = inner, states, taps

    def new_state(self, n):
        """What a sequence carries from token to token: K-1 rows of the convolution, the scan's state."""
        w = self.p["conv_w"]
        return (torch.zeros(n, self.taps - 1, self.inner, dtype=w.dtype, device=w.device),
                torch.zeros(n, self.inner, self.states, device=w.device))

    def forward(self, x, state=None, lengths=None, keep=None):
        """x [N,L,C] -> (y [N,L,C], the state after each sequence's last valid token).
        keep: a dict that takes what backward needs."""
        p, d, s = self.p, self.inner, self.states
        conv_state, scan_state = (None, None) if state is None else state
        h, mean, rstd = cn.layer_norm(x, p["norm_w"], p["norm_b"], return_stats=True)
        vz = project(h, p["w_in"])
        u, conv_state = cn.causal_conv1d(vz[..., :d], p["conv_w"], p["conv_b"], activation="silu", state=conv_state,
                                         lengths=lengths, return_state=True)
        r = project(u, p["w_rank"])
        delta, bc, a = project(r, p["w_delta"]), project(u, p["w_bc"]), -torch.exp(p["a_log"])
        y, scan_state = cn.selective_scan(u, delta, a, bc[..., :s], bc[..., s:], skip=p["skip"], gate=vz[..., d:],
                                          delta_bias=p["delta_bias"], softplus=True, state=scan_state,
                                          lengths=lengths, return_state=True)
        if keep is not None:
            keep.update(x=x, mean=mean, rstd=rstd, h=h, vz=vz, u=u, r=r, delta=delta, bc=bc, a=a, y=y,
                        lengths=lengths)
        return x + project(y, p["w_out"]), (conv_state, scan_state)

    def step(self, x, state):
        """One new token x [N,C] of every sequence; state moves on in place."""
        p, d, s = self.p, self.inner, self.states
        row = lambda t, w: project(t[:, None], w)[:, 0]
        h = cn.layer_norm(x, p["norm_w"], p["norm_b"])
        vz = row(h, p["w_in"])
        u = cn.causal_conv1d_step(vz[:, :d], state[0], p["conv_w"], p["conv_b"], activation="silu")
        delta, bc = row(row(u, p["w_rank"]), p["w_delta"]), row(u, p["w_bc"])
        y = cn.selective_scan_step(u, delta, -torch.exp(p["a_log"]), bc[:, :s], bc[:, s:], state[1], skip=p["skip"],
                                   gate=vz[:, d:], delta_bias=p["delta_bias"], softplus=True)
        return x + row(y, p["w_out"])

    def backward(self, dout, k):
        """(dx, gradients by parameter name) of forward(..., keep=k) without an initial state."""
        p, d, s, g = self.p, self.inner, self.states, {}
        dy, g["w_out"] = project_backward(dout, k["y"], p["w_out"])
        scan = cn.selective_scan_backward(dy, k["u"], k["delta"], k["a"], k["bc"][..., :s], k["bc"][..., s:],
                                          skip=p["skip"], gate=k["vz"][..., d:], delta_bias=p["delta_bias"],
                                          softplus=True, lengths=k["lengths"])
        g["a_log"], g["skip"], g["delta_bias"] = scan.a * k["a"], scan.skip, scan.delta_bias
        dr, g["w_delta"] = project_backward(scan.delta, k["r"], p["w_delta"])
        du_rank, g["w_rank"] = project_backward(dr, k["u"], p["w_rank"])
        du_bc, g["w_bc"] = project_backward(torch.cat([scan.b, scan.c], -1), k["u"], p["w_bc"])
        conv = cn.causal_conv1d_backward(scan.u + du_rank + du_bc, k["vz"][..., :d], p["conv_w"], p["conv_b"],
                                         activation="silu", lengths=k["lengths"])
        g["conv_w"], g["conv_b"] = conv.w, conv.bias
        dh, g["w_in"] = project_backward(torch.cat([conv.x, scan.gate], -1), k["h"], p["w_in"])
        dx, g["norm_w"], g["norm_b"] = cn.layer_norm_backward(dh, k["x"], k["mean"], k["rstd"], p["norm_w"])
        return dx + dout, g


def answer(block, prompts, lengths, tokens):
    """Prompts of several lengths in one call, then `tokens` [N,T,C] one by one; the outputs of both."""
    y, state = block.forward(prompts, lengths=lengths)
    return y, torch.stack([block.step(tokens[:, t].contiguous(), state) for t in range(tokens.shape[1])], 1)


def train(block, steps=40, rate=0.02, seed=1, report=None):
    """Learns to give back the input of three positions earlier, with steps scaled by
    running means of the gradients and their squares (Adam); the losses."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    losses = []
    mean = {k: torch.zeros_like(t) for k, t in block.p.items()}
    square = {k: torch.zeros_like(t) for k, t in block.p.items()}
    for i in range(steps):
        x = torch.randn(4, 64, block.p["norm_w"].numel(), generator=g, device="cuda")
        x = x.to(block.p["norm_w"].dtype)
        want = torch.zeros_like(x)
        want[:, 3:] = x[:, :-3]
        keep = {}
        y, _ = block.forward(x, keep=keep)
        diff = (y - x) - want
        losses.append(float((diff.float() ** 2).mean()))
        _, grads = block.backward(diff * (2.0 / diff[..., 0].numel()), keep)
        for name, t in block.p.items():
            m, q = mean[name].lerp_(grads[name], 0.1), square[name].lerp_(grads[name] ** 2, 0.01)
            t -= rate * (m / (1 - 0.9 ** (i + 1))) / ((q / (1 - 0.99 ** (i + 1))).sqrt() + 1e-8)
        if report and i % 10 == 0:
            report(f"step {i}: loss {losses[-1]:.4f}")
    return losses


def main():
    torch.manual_seed(0)
    block = SequenceBlock(512, 1024)
    lengths = torch.tensor([200, 1, 77, 0], dtype=torch.int32, device="cuda")
    x = torch.randn(4, 208, 512, device="cuda").bfloat16()
    _, by_token = answer(block, x[:, :200].contiguous(), lengths, x[:, 200:])
    # the same tokens behind the first prompt as one longer prompt
    whole, _ = block.forward(x[:1])
    far = (whole[0, 200:].float() - by_token[0].float()).abs().max() / whole.float().abs().max()
    print(f"a prompt of 200 and 8 tokens against one of 208: largest difference {float(far):.1e} of the largest output")
    losses = train(SequenceBlock(64, 128, dtype=torch.float32), report=print)
    print(f"training: loss {losses[0]:.4f} -> {losses[-1]:.4f}")


if __name__ == "__main__":
    main()
