"""The root-mean-square norm, rotary positions and linear attention together, as a residual
block uses them with the package's pointwise conv1d:

    h = rms_norm(x + r)                     the residual stream goes on as x + r
    q, k, v = parts of one projection's rows, q and k turned by their positions in place
    y = rms_norm(linear_attention(q, k, v))  over each head
    out = projection(y)

on ragged prompts, token by token, and backwards, against the same block in 64 bits."""
import math

import pytest
import torch

import attention_reference as A

pytestmark = pytest.mark.gpu

cn = pytest.importorskip("convolution_nhwc_conv2d_amd")

C, H, DK, DV, R = 96, 3, 32, 40, 24
EPS = 1e-6


def _project(x, w):
    return cn.conv1d(x, w[:, None, :])


class Block:
    def __init__(self, dtype, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        r = lambda *s, scale=1.0: (torch.randn(*s, generator=g, device="cuda") * scale).to(dtype)
        self.wide = H * (2 * DK + DV)
        self.norm, self.head_norm = 1 + r(C, scale=0.1), 1 + r(DV, scale=0.1)
        self.w_in, self.w_out = r(self.wide, C, scale=C ** -0.5), r(C, H * DV, scale=(H * DV) ** -0.5)
        self.log_decay = -torch.tensor([0.5, 0.05, 0.002], device="cuda")
        self.freqs = cn.rotary_frequencies(R, scaling="yarn", factor=4.0, original_length=64)
        self.scale = 0.1 * math.log(4.0) + 1

    def parts(self, p):
        qk, v = p[..., :2 * H * DK].unflatten(-1, (2 * H, DK)), p[..., 2 * H * DK:].unflatten(-1, (H, DV))
        return qk, v

    def forward(self, x, res, state=None, lengths=None, keep=None):
        h, z, rstd = cn.rms_norm(x, self.norm, EPS, residual=res, return_stats=True)
        p = _project(h, self.w_in)
        qk, v = self.parts(p)
        cn.rotary(qk, self.freqs, scale=self.scale, out=qk)  # in place, inside the projection's rows
        y, state = cn.linear_attention(qk[..., :H, :], qk[..., H:, :], v, self.log_decay, scale=DK ** -0.5, state=state,
                                       lengths=lengths, return_state=True)
        u, urstd = cn.rms_norm(y, self.head_norm, EPS, return_stats=True)
        if keep is not None:
            keep.update(h=h, z=z, rstd=rstd, p=p, y=y, urstd=urstd, u=u, lengths=lengths)
        return _project(u.flatten(-2), self.w_out), z, state

    def step(self, x, res, state, at):
        h, z = cn.rms_norm(x, self.norm, EPS, residual=res, sum_out=res)
        qk, v = self.parts(_project(h[:, None], self.w_in)[:, 0])
        cn.rotary(qk, self.freqs, positions=at, scale=self.scale, out=qk)
        y = cn.linear_attention_step(qk[:, :H], qk[:, H:], v, self.log_decay, state, scale=DK ** -0.5)
        u = cn.rms_norm(y, self.head_norm, EPS)
        return _project(u.flatten(-2)[:, None], self.w_out)[:, 0], z

    def backward(self, dout, dz, k):
        rows = lambda t: t.reshape(-1, t.shape[-1])
        weight = lambda dy, x: _project(rows(x).t().contiguous()[None], rows(dy).t().contiguous())[0].t().contiguous()
        g = {"w_out": weight(dout, k["u"].flatten(-2))}
        du = _project(dout, self.w_out.t().contiguous()).unflatten(-1, (H, DV))
        dy, g["head_norm"] = cn.rms_norm_backward(du, k["y"], k["urstd"], self.head_norm)
        qk, v = self.parts(k["p"])
        r = cn.linear_attention_backward(dy, qk[..., :H, :], qk[..., H:, :], v, self.log_decay, scale=DK ** -0.5,
                                         lengths=k["lengths"], decay_grad=True)
        g["log_decay"] = r.log_decay
        dqk = cn.rotary_backward(torch.cat([r.q, r.k], -2), self.freqs, scale=self.scale)
        dp = torch.cat([dqk.flatten(-2), r.v.flatten(-2)], -1)
        g["w_in"] = weight(dp, k["h"])
        dx, g["norm"] = cn.rms_norm_backward(_project(dp, self.w_in.t().contiguous()), k["z"], k["rstd"], self.norm,
                                             dsum=dz)
        return dx, g

    def plain(self, x, res, p, lengths):
        """The block of 64-bit tensors p, differentiable: all positions with all positions."""
        n, l = x.shape[:2]
        norm = lambda t, w: t * (t.square().mean(-1, keepdim=True) + EPS) ** -0.5 * w
        z = x + res
        rows = norm(z, p["norm"]) @ p["w_in"].t()
        qk, v = self.parts(rows)
        t = torch.arange(l, device="cuda")
        angle = t[:, None, None] * self.freqs
        c, s, half = torch.cos(angle) * self.scale, torch.sin(angle) * self.scale, R // 2
        a, b = qk[..., :half], qk[..., half:R]
        qk = torch.cat([a * c - b * s, a * s + b * c, qk[..., R:]], -1)
        m = torch.full((n,), l, device="cuda") if lengths is None else lengths.long()
        live = (t < m[:, None])[..., None, None]
        q, k = torch.where(live, qk[..., :H, :], 0.0), torch.where(live, qk[..., H:, :], 0.0)
        far = (t[:, None] - t).double()
        between = torch.where(far >= 0, torch.exp(p["log_decay"][:, None, None] * far.clamp(min=0)), 0.0)
        y = torch.einsum("nuhd,nshd,hus,nshe->nuhe", q, k, between, v) * DK ** -0.5
        return norm(y, p["head_norm"]).flatten(-2) @ p["w_out"].t(), z

    def leaves(self):
        return {n: getattr(self, n).double().requires_grad_() for n in ("norm", "head_norm", "w_in", "w_out", "log_decay")}


def _data(dtype, seed, n, l):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [torch.randn(n, l, C, generator=g, device="cuda").to(dtype) for _ in range(4)]


# Off by the roundings of the activations on the way, each u relative to a value whose
# size the next norm or product keeps: about ten of them, on rows of random signs; the
# norm of a whole tensor's difference stays below 16 u (bf16, f16).  fp32: sums of a
# few hundred terms and more, 2^-24 each, below 2^-16.
BOUND = {torch.float32: 2.0 ** -16, torch.float16: 16 * 2.0 ** -11, torch.bfloat16: 16 * 2.0 ** -8}


def _near(got, want, dtype, what):
    d = (got.double() - want).norm() / want.norm()
    assert float(d) < BOUND[dtype], f"{what}: {float(d)}"


@pytest.mark.parametrize("dtype", list(BOUND))
@pytest.mark.parametrize("lengths", [None, [150, 1, 0, 77]])
def test_block_and_its_gradient(dtype, lengths):
    block = Block(dtype)
    n = 2 if lengths is None else len(lengths)
    x, res, dout, dz = _data(dtype, 1, n, 150)
    m = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
    keep = {}
    out, z, _ = block.forward(x, res, lengths=m, keep=keep)
    dx, g = block.backward(dout, dz, keep)
    p = block.leaves()
    x64 = x.double().requires_grad_()
    want, wz = block.plain(x64, res.double(), p, m)
    _near(out, want.detach(), dtype, "out")
    _near(z, wz.detach(), dtype, "sum")
    grads = torch.autograd.grad((want * dout.double()).sum() + (wz * dz.double()).sum(), [x64] + list(p.values()))
    _near(dx, grads[0], dtype, "dx")
    for name, w in zip(p, grads[1:]):
        _near(g[name], w, dtype, name)


def test_tokens_follow_ragged_prompts():
    """Prompts of several lengths in one call, then tokens of all sequences with positions of their own: what each
    sequence gives alone."""
    block = Block(torch.float32)
    lengths = torch.tensor([40, 1, 17, 0], dtype=torch.int32, device="cuda")
    x, res, tok, tres = _data(torch.float32, 2, 4, 40)
    _, _, state = block.forward(x, res, lengths=lengths)
    at, outs = lengths.clone(), []
    for t in range(5):
        r = tres[:, t].contiguous()
        out, z = block.step(tok[:, t].contiguous(), r, state, at)
        assert z.data_ptr() == r.data_ptr()
        outs.append(out)
        at += 1
    p = {k: v.detach() for k, v in block.leaves().items()}
    for n, m in enumerate([40, 1, 17, 0]):
        xs = torch.cat([x[n, :m], tok[n, :5]])[None].double()
        rs = torch.cat([res[n, :m], tres[n, :5]])[None].double()
        want, _ = block.plain(xs, rs, p, None)
        _near(torch.stack(outs, 1)[n], want[0, m:], torch.float32, f"sequence {n}")


def test_the_block_in_a_graph():
    block = Block(torch.bfloat16)
    x, res, dout, dz = _data(torch.bfloat16, 3, 2, 200)

    def step():
        keep = {}
        out, z, state = block.forward(x, res, keep=keep)
        dx, g = block.backward(dout, dz, keep)
        return [out, z, state, dx] + [g[k] for k in sorted(g)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        want = step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(3):
        for t in got:
            t.zero_()
        graph.replay()
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
