"""Measured cases of the operators of a linear attention block: root-mean-square
norm (with the residual's addition, with an output in 8 bits, backward), rotary
positions (both layouts, backward) and linear attention with a decay for each
head (prompts, backward, single tokens).

``run`` has two forms.  With ``own`` false it computes the operator from its
formula with elementary torch operations in 32 bits (angles, and decays by their
distance, in 64), rounded once at the end; with ``own`` true it calls the
package.  ``exact`` computes the same outputs in 64 bits, apart from both: the
norm's gradient there is automatic differentiation, the rotation a product of
complex numbers, and linear attention runs token by token, where the plain form
has one product of all positions with all positions.

Formulas (n: sequence, t, u, s: position, h: head, c or d: channel):

  RMS norm          z = x + residual, y = z * rstd * w, rstd = 1 / sqrt(mean z^2 + eps)
                    8 bits: y = q * scale, scale = max |y| / 448 of the row or of each
                    group of channels, at least 2^-100; q in e4m3
  rotary            angle = position * frequency[i]; the channels i and i + R/2 (half) or
                    2i and 2i + 1 (interleaved) of every head turn by it, times scale;
                    the channels from R on stay
  linear attention  S[t] = exp(log_decay) S[t-1] + k[t]^T v[t],  y[t] = scale q[t] S[t]

``lengths`` gives each sequence's valid positions; past them outputs and
gradients are 0 and the state stands still.
"""
import math

import torch

own = False

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
EPS = 1e-6
F8_MAX, SCALE_MIN = 448.0, 2.0 ** -100

# ------------------------------------------------------------------ cases


def listed():
    return [
        # one token's activations and its residual between the layers of a model that is answering
        {"name": "rms-one-token", "kind": "rms", "dtype": "bf16", "n": 1, "l": 1, "c": 512, "residual": True},
        # prompts' activations with the residual stream, wide rows
        {"name": "rms-residual", "kind": "rms", "dtype": "bf16", "n": 4, "l": 4096, "c": 4096, "residual": True},
        # the same rows on their way into a product in 8 bits, scales for every 128 channels
        {"name": "rms-8bit", "kind": "rms_8bit", "dtype": "bf16", "n": 4, "l": 4096, "c": 4096, "residual": True,
         "group": 128},
        # an odd count of rows whose width fills no power of two, one scale a row
        {"name": "rms-8bit-odd", "kind": "rms_8bit", "dtype": "f16", "n": 1, "l": 3001, "c": 1000, "residual": False,
         "group": 0},
        # a training step, the gradient of the residual stream joining
        {"name": "rms-grad", "kind": "rms_grad", "dtype": "bf16", "n": 8, "l": 2048, "c": 2048, "residual": True},
        # queries' and keys' heads of prompts as they lie in a projection's rows
        {"name": "rotary-prompt", "kind": "rotary", "dtype": "bf16", "n": 4, "l": 4096, "h": 32, "d": 128, "r": 128,
         "interleaved": False, "split": True, "far": 0},
        # new tokens far along their sequences, the first half of each head turned
        {"name": "rotary-token-far", "kind": "rotary_token", "dtype": "f16", "n": 64, "h": 40, "d": 128, "r": 64,
         "interleaved": True, "split": True, "far": 1000000},
        # a training step's gradient in 32 bits, odd sizes
        {"name": "rotary-grad-odd", "kind": "rotary_grad", "dtype": "f32", "n": 3, "l": 1023, "h": 15, "d": 80, "r": 80,
         "interleaved": True, "split": False, "far": 0},
        # one long prompt
        {"name": "attention-long", "kind": "attn", "dtype": "bf16", "n": 1, "l": 16384, "h": 16, "dk": 128, "dv": 128,
         "split": True, "ragged": False, "state": False},
        # prompts of several lengths that go on from their states, in 32 bits
        {"name": "attention-ragged", "kind": "attn", "dtype": "f32", "n": 6, "l": 1023, "h": 5, "dk": 64, "dv": 96,
         "split": False, "ragged": True, "state": True},
        # a training step
        {"name": "attention-grad", "kind": "attn_grad", "dtype": "bf16", "n": 8, "l": 2048, "h": 16, "dk": 128,
         "dv": 128, "split": True, "ragged": False, "state": False, "decay": True},
        # one new token of each of 64 sequences
        {"name": "attention-token", "kind": "attn_step", "dtype": "bf16", "n": 64, "h": 16, "dk": 128, "dv": 128},
    ]


def _log(rng, lo, hi):
    """An integer of [lo, hi], spread over the logarithm, odd and even ones alike."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    kind = rng.choice(["rms", "rms_8bit", "rms_grad", "rotary", "rotary_token", "rotary_grad", "attn", "attn",
                       "attn_grad", "attn_step"])
    case = {"kind": kind, "dtype": rng.choice(["f32", "f16", "bf16"])}
    if kind.startswith("rms"):
        group = rng.choice([0, 32, 64, 128]) if kind == "rms_8bit" else 0
        c = _log(rng, 32, 8192)
        if group:
            c = group * max(1, c // group)
        n = _log(rng, 1, 8)
        case.update(n=n, l=_log(rng, 1, max(1, min(8192, (1 << 25) // (c * n)))), c=c, residual=rng.random() < 0.6)
        return {**case, "group": group} if kind == "rms_8bit" else case
    if kind.startswith("rotary"):
        n, h, d = _log(rng, 1, 8), _log(rng, 1, 40), 2 * _log(rng, 8, 128)
        r = d if rng.random() < 0.5 else 2 * rng.randint(1, d // 2)
        flags = {"r": r, "interleaved": rng.random() < 0.5, "split": rng.random() < 0.5,
                 "far": rng.choice([0, 0, 1000000])}
        if kind == "rotary_token":
            return {**case, "n": _log(rng, 1, 128), "h": h, "d": d, **flags}
        return {**case, "n": n, "l": _log(rng, 1, max(1, min(8192, (1 << 25) // (n * h * d)))), "h": h, "d": d, **flags}
    h = _log(rng, 1, 24)
    dk, dv = (rng.choice([16, 32, 48, 64, 64, 80, 96, 128, 128, 100, 192, 256]) for _ in range(2))
    if kind == "attn_step":
        return {**case, "n": _log(rng, 1, 96), "h": h, "dk": dk, "dv": dv}
    n = _log(rng, 1, 8)
    # what every position does with every other one, in the plain form, and what a state takes
    l = _log(rng, 1, max(1, min(8192, int(math.sqrt((1 << 29) / (n * h))))))
    case.update(n=n, l=l, h=h, dk=dk, dv=dv, split=rng.random() < 0.5, ragged=rng.random() < 0.5,
                state=rng.random() < 0.5)
    return {**case, "decay": rng.random() < 0.5} if kind == "attn_grad" else case


def work(case):
    e, kind = SIZE[case["dtype"]], case["kind"]
    if kind.startswith("rms"):
        rows, c, more = case["n"] * case["l"], case["c"], 1 if case["residual"] else 0
        if kind == "rms":  # x, residual, w read; y, the sum, rstd written
            return {"bytes": e * (2 * (1 + more) * rows * c + c) + 4 * rows, "flops": (4 + more) * rows * c}
        if kind == "rms_8bit":
            groups = c // case["group"] if case["group"] else 1
            return {"bytes": e * ((1 + 2 * more) * rows * c + c) + rows * c + 4 * rows * groups,
                    "flops": (6 + more) * rows * c}
        return {"bytes": e * ((3 + more) * rows * c + 2 * c) + 4 * rows, "flops": (9 + more) * rows * c}
    if kind.startswith("rotary"):
        tokens = case["n"] * case.get("l", 1)
        return {"bytes": 2 * e * tokens * case["h"] * case["d"] + 4 * tokens + 4 * case["r"],
                "flops": 3 * tokens * case["h"] * case["r"]}
    n, h, dk, dv = (case[k] for k in ("n", "h", "dk", "dv"))
    if kind == "attn_step":
        return {"bytes": 8 * n * h * dk * dv + e * n * h * (2 * dk + 2 * dv) + 4 * h, "flops": 5 * n * h * dk * dv}
    live = sum(_lengths(case)) if case["ragged"] else n * case["l"]
    state = 4 * n * h * dk * dv
    if kind == "attn":  # q, k, v read, y written; by the recurrence 4 operations to an element of the state
        return {"bytes": e * h * (live * (2 * dk + dv) + n * case["l"] * dv) + (2 if case["state"] else 1) * state,
                "flops": 4 * live * h * dk * dv}
    return {"bytes": e * h * (live * (2 * dk + 2 * dv) + n * case["l"] * (2 * dk + dv))
            + (3 * state if case["state"] else 0), "flops": (12 if case["decay"] else 10) * live * h * dk * dv}


# ------------------------------------------------------------------ inputs


def _lengths(case):
    """Valid positions: one full sequence, one of a single token, one of none, the rest between."""
    n, l = case["n"], case["l"]
    fixed = [l, 1, 0]
    return [fixed[i] if i < 3 else 1 + (i * 7919 + l // 2) % l for i in range(n)]


def _inputs(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1000003 + 29)
    dt, kind = DT[case["dtype"]], case["kind"]

    def normal(*shape, scale=1.0, shift=0.0, dtype=dt):
        return (torch.randn(shape, generator=g, device="cuda") * scale + shift).to(dtype)

    if kind.startswith("rms"):
        shape = (case["n"], case["l"], case["c"])
        st = {"x": normal(*shape, scale=1.5), "w": normal(case["c"], scale=0.1, shift=1.0), "residual": None,
              "group": case.get("group", 0)}
        if kind == "rms_grad":
            st["dy"] = normal(*shape)
            st["dsum"] = normal(*shape) if case["residual"] else None
            # the statistics that the forward pass left
            st["rstd"] = (st["x"].float().square().mean(-1) + EPS).rsqrt()
        elif case["residual"]:
            st["residual"] = normal(*shape, scale=4.0)
        return st
    if kind.startswith("rotary"):
        n, h, d = case["n"], case["h"], case["d"]
        lead = (n,) if kind == "rotary_token" else (n, case["l"])
        if case["split"]:  # the first heads of a wider projection's rows
            x = normal(*lead, (h + 2) * d)[..., :h * d].unflatten(-1, (h, d))
        else:
            x = normal(*lead, h, d)
        i = torch.arange(case["r"] // 2, device="cuda", dtype=torch.float64)
        st = {"x": x, "freqs": 10000.0 ** (-2.0 * i / case["r"]), "interleaved": case["interleaved"],
              "positions": None, "scale": 1.0}
        if case["far"] or kind == "rotary_token":
            at = torch.randint(0, max(4096, case["far"]), lead[:1], generator=g, device="cuda", dtype=torch.int32)
            st["positions"] = at if kind == "rotary_token" else (
                at[:, None] + torch.arange(case["l"], device="cuda", dtype=torch.int32))
        return st
    n, h, dk, dv = (case[k] for k in ("n", "h", "dk", "dv"))
    # decays whose half-lives go from 4 to 4096 positions over the heads
    life = torch.exp(torch.rand(h, generator=g, device="cuda") * math.log(1024.0)) * 4.0
    st = {"log_decay": -math.log(2.0) / life, "scale": dk ** -0.5, "lengths": None, "state": None,
          "dstate": None, "decay": case.get("decay", False)}
    if kind == "attn_step":
        st.update(q=normal(n, h, dk), k=normal(n, h, dk), v=normal(n, h, dv),
                  state=normal(n, h, dk, dv, dtype=torch.float32))
        st["new_state"] = torch.empty_like(st["state"])
        return st
    l = case["l"]
    if case["split"]:  # parts of one projection's rows
        rows = normal(n, l, h * (2 * dk + dv))
        st.update(q=rows[..., :h * dk].unflatten(-1, (h, dk)), k=rows[..., h * dk:2 * h * dk].unflatten(-1, (h, dk)),
                  v=rows[..., 2 * h * dk:].unflatten(-1, (h, dv)))
    else:
        st.update(q=normal(n, l, h, dk), k=normal(n, l, h, dk), v=normal(n, l, h, dv))
    if case["ragged"]:
        st["lengths"] = torch.tensor(_lengths(case), dtype=torch.int32, device="cuda")
    if case["state"]:
        st["state"] = normal(n, h, dk, dv, dtype=torch.float32)
    if kind == "attn_grad":
        st["dy"] = normal(n, l, h, dv)
        if case["state"]:
            st["dstate"] = normal(n, h, dk, dv, scale=0.1, dtype=torch.float32)
    return st


def prepare(case, seed):
    st = _inputs(case, seed)
    st["kind"] = case["kind"]
    return st


# ------------------------------------------------------------------ one pass


def run(st):
    return (_run_own if own else _run_plain)(st)


def _run_own(st):
    import convolution_nhwc_conv2d_amd as cn
    kind = st["kind"]
    if kind == "rms":
        return cn.rms_norm(st["x"], st["w"], EPS, residual=st["residual"], return_stats=True)
    if kind == "rms_8bit":
        return cn.rms_norm_quantized(st["x"], st["w"], EPS, group=st["group"] or None, residual=st["residual"])
    if kind == "rms_grad":
        return cn.rms_norm_backward(st["dy"], st["x"], st["rstd"], st["w"], dsum=st["dsum"])
    if kind in ("rotary", "rotary_token"):
        return cn.rotary(st["x"], st["freqs"], positions=st["positions"], interleaved=st["interleaved"],
                         scale=st["scale"])
    if kind == "rotary_grad":
        return cn.rotary_backward(st["x"], st["freqs"], positions=st["positions"], interleaved=st["interleaved"],
                                  scale=st["scale"])
    if kind == "attn":
        return cn.linear_attention(st["q"], st["k"], st["v"], st["log_decay"], scale=st["scale"], state=st["state"],
                                   lengths=st["lengths"], return_state=True)
    if kind == "attn_grad":
        r = cn.linear_attention_backward(st["dy"], st["q"], st["k"], st["v"], st["log_decay"], scale=st["scale"],
                                         state=st["state"], lengths=st["lengths"], dstate=st["dstate"],
                                         decay_grad=st["decay"])
        return [t for t in (r.q, r.k, r.v, r.log_decay, r.state) if t is not None]
    y = cn.linear_attention_step(st["q"], st["k"], st["v"], st["log_decay"], st["state"], scale=st["scale"],
                                 state_out=st["new_state"])
    return y, st["new_state"]


def _run_plain(st):
    kind = st["kind"]
    if kind == "rms":
        z, rstd, y = _plain_rms(st)
        dt = st["x"].dtype
        return (y.to(dt), rstd) if st["residual"] is None else (y.to(dt), z.to(dt), rstd)
    if kind == "rms_8bit":
        z, _, y = _plain_rms(st)
        groups = y.unflatten(-1, (-1, st["group"] or y.shape[-1]))
        scale = torch.clamp(groups.abs().amax(-1) / F8_MAX, min=SCALE_MIN)
        q = (groups / scale[..., None]).flatten(-2).to(torch.float8_e4m3fn)
        scale = scale if st["group"] else scale[..., 0]
        return (q, scale) if st["residual"] is None else (q, scale, z.to(st["x"].dtype))
    if kind == "rms_grad":
        x, dy, rstd = st["x"].float(), st["dy"].float(), st["rstd"][..., None]
        xh, g = x * rstd, dy * st["w"].float()
        dx = rstd * (g - xh * (g * xh).mean(-1, keepdim=True))
        if st["dsum"] is not None:
            dx = dx + st["dsum"].float()
        return dx.to(st["x"].dtype), (dy * xh).sum((0, 1)).to(st["w"].dtype)
    if kind.startswith("rotary"):
        return _plain_rotary(st, -1.0 if kind == "rotary_grad" else 1.0)
    if kind == "attn":
        return _plain_attention(st)
    if kind == "attn_grad":
        return _plain_attention_grad(st)
    q, k, v = st["q"].float(), st["k"].float(), st["v"].float()
    s = torch.exp(st["log_decay"])[:, None, None] * st["state"] + k[..., None] * v[..., None, :]
    st["new_state"].copy_(s)
    return (st["scale"] * (q[..., None] * s).sum(-2)).to(st["v"].dtype), st["new_state"]


def _plain_rms(st):
    z = st["x"].float()
    if st["residual"] is not None:
        z = z + st["residual"].float()
    rstd = 1.0 / torch.sqrt((z * z).mean(-1, keepdim=True) + EPS)
    return z, rstd[..., 0], z * rstd * st["w"].float()


def _plain_rotary(st, sign):
    x, freqs = st["x"], st["freqs"]
    at = st["positions"]
    if at is None:
        at = torch.arange(x.shape[1], device="cuda")[None, :]
    angle = at.double()[..., None] * freqs * sign
    cos, sin = ((f(angle) * st["scale"]).float()[..., None, :] for f in (torch.cos, torch.sin))
    half = freqs.shape[0]
    turned, rest = x[..., :2 * half].float(), x[..., 2 * half:]
    if st["interleaved"]:
        a, b = turned[..., 0::2], turned[..., 1::2]
        out = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    else:
        a, b = turned[..., :half], turned[..., half:]
        out = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    return torch.cat([out.to(x.dtype), rest], -1)


def _powers(st, far):
    """decay^0 ... decay^far of every head, [H, far + 1]."""
    return torch.exp(st["log_decay"].double()[:, None] * torch.arange(far + 1, device="cuda")).float()


def _plain_terms(st):
    """q, k, v [N,H,L,D] (0 past the lengths), decay^(u-s) for u >= s and 0 otherwise
    [H,L,L], decay^(t+1) [H,L], decay^(length-1-t) [N,H,L] and decay^length [N,H]."""
    q, k, v = (st[x].float().transpose(1, 2) for x in "qkv")
    n, h, l, _ = q.shape
    t = torch.arange(l, device="cuda")
    lengths = torch.full((n,), l, device="cuda") if st["lengths"] is None else st["lengths"].long()
    valid = (t < lengths[:, None])[:, None, :, None]
    zero = torch.zeros((), device="cuda")
    q, k, v = (torch.where(valid, x, zero).contiguous() for x in (q, k, v))
    power = _powers(st, l)
    far = t[:, None] - t
    between = power[:, far.clamp(min=0)] * (far >= 0)
    ahead = lengths[:, None] - 1 - t
    to_end = power[:, ahead.clamp(min=0)].transpose(0, 1) * (ahead >= 0)[:, None]
    return q, k, v, valid, between, power[:, 1:], to_end, power[:, lengths].t()


def _back(t, dt):
    return t.transpose(1, 2).to(dt).contiguous()


def _plain_attention(st):
    q, k, v, valid, between, before, to_end, whole = _plain_terms(st)
    p = torch.matmul(q, k.transpose(-1, -2).contiguous())
    p *= between
    y = torch.matmul(p, v)
    state = torch.matmul((k * to_end[..., None]).transpose(-1, -2).contiguous(), v)
    if st["state"] is not None:
        y = y + before[..., None] * torch.matmul(q, st["state"])
        state = state + whole[..., None, None] * st["state"]
    return _back(torch.where(valid, y * st["scale"], torch.zeros((), device="cuda")), st["q"].dtype), state


def _plain_attention_grad(st):
    q, k, v, valid, between, before, to_end, whole = _plain_terms(st)
    dt, l = st["q"].dtype, q.shape[2]
    t = torch.arange(l, device="cuda")
    zero = torch.zeros((), device="cuda")
    dy = torch.where(valid, st["dy"].float().transpose(1, 2), zero).contiguous() * st["scale"]
    p = torch.matmul(q, k.transpose(-1, -2).contiguous()) * between
    dp = torch.matmul(dy, v.transpose(-1, -2).contiguous())
    if st["decay"]:
        dg = (p * dp * (t[:, None] - t)).double().sum((0, 2, 3))
    dp *= between
    dq = torch.matmul(dp, k)
    dk = torch.matmul(dp.transpose(-1, -2).contiguous(), q)
    dv = torch.matmul(p.transpose(-1, -2).contiguous(), dy)
    dstate = None
    if st["state"] is not None:  # what goes through the state at the start and the one at the end
        s0, ds = st["state"], st["dstate"]
        more_q = before[..., None] * torch.matmul(dy, s0.transpose(-1, -2).contiguous())
        more_k = to_end[..., None] * torch.matmul(v, ds.transpose(-1, -2).contiguous())
        dq, dk, dv = dq + more_q, dk + more_k, dv + to_end[..., None] * torch.matmul(k, ds)
        dstate = torch.matmul((q * before[..., None]).transpose(-1, -2).contiguous(), dy)
        dstate = dstate + whole[..., None, None] * ds
        if st["decay"]:
            lengths = torch.full((q.shape[0],), l, device="cuda") if st["lengths"] is None else st["lengths"].long()
            dg = dg + ((q * more_q).sum(-1) * (t + 1)).double().sum((0, 2))
            dg = dg + ((k * more_k).sum(-1) * (lengths[:, None, None] - 1 - t)).double().sum((0, 2))
            dg = dg + ((s0 * ds).double().sum((-1, -2)) * whole * lengths[:, None]).sum(0)
    out = [_back(torch.where(valid, x, zero), dt) for x in (dq, dk, dv)]
    if st["decay"]:
        out.append(dg.float())
    return out + ([dstate] if dstate is not None else [])


# ------------------------------------------------------------------ 64 bits


def _e4m3(v):
    """The nearest value that e4m3 holds, ties to the even one."""
    _, e = torch.frexp(v)
    step = torch.exp2((torch.clamp(e, min=-5) - 4).double())  # 3 bits behind the leading one; subnormals below 2^-6
    return torch.clamp(torch.round(v / step) * step, -F8_MAX, F8_MAX)


def exact(case, seed):
    st = _inputs(case, seed)
    kind = case["kind"]
    leaf = {k: v.double() if torch.is_tensor(v) and v.is_floating_point() else v for k, v in st.items()}
    if kind == "rms_grad":
        # the statistics are the forward pass's, so they are functions of x here
        x, w = leaf["x"].requires_grad_(), leaf["w"].requires_grad_()
        dx, dw = torch.autograd.grad(x * (x.pow(2).mean(-1, keepdim=True) + EPS) ** -0.5 * w, (x, w), leaf["dy"])
        return dx if leaf["dsum"] is None else dx + leaf["dsum"], dw
    if kind.startswith("rms"):
        z = leaf["x"] if leaf["residual"] is None else leaf["x"] + leaf["residual"]
        rstd = (torch.linalg.vector_norm(z, dim=-1) ** 2 / case["c"] + EPS) ** -0.5
        y = torch.einsum("nlc,nl,c->nlc", z, rstd, leaf["w"])
        more = () if leaf["residual"] is None else (z,)
        if kind == "rms":
            return (y,) + more + (rstd,)
        rows = y.reshape(case["n"], case["l"], -1, case["group"] or case["c"])
        scale = torch.maximum(rows.max(-1).values, -rows.min(-1).values) / F8_MAX
        scale = torch.clamp(scale, min=SCALE_MIN)
        q = _e4m3(rows / scale[..., None]).reshape(y.shape)
        return (q, scale if case["group"] else scale.squeeze(-1)) + more
    if kind.startswith("rotary"):
        x, r = leaf["x"], case["r"]
        at = torch.arange(x.shape[1], device="cuda")[None] if leaf["positions"] is None else leaf["positions"]
        angle = at[..., None, None] * leaf["freqs"]
        turn = torch.polar(torch.full_like(angle, leaf["scale"]), -angle if kind == "rotary_grad" else angle)
        part = x[..., :r].unflatten(-1, (-1, 2) if case["interleaved"] else (2, -1))
        axis = -1 if case["interleaved"] else -2
        z = torch.complex(*part.unbind(axis)) * turn
        return torch.cat([torch.stack([z.real, z.imag], axis).flatten(-2), x[..., r:]], -1)
    return _exact_attention(case, leaf)


def _exact_attention(case, leaf):
    """Token by token; the backward pass along the positions from the end.  With
    T[t] = decay (T[t-1] + S[t-1]), the state's derivative by log_decay, the decay's
    gradient is the sum of scale dy q T and, at the end, dstate T."""
    kind = case["kind"]
    one = kind == "attn_step"
    seq = [n for n in ("q", "k", "v", "dy") if n in leaf]
    x = {n: (leaf[n][:, None] if one else leaf[n]).movedim(1, 0) for n in seq}
    decay = torch.exp(leaf["log_decay"])[:, None, None]
    n, h, dk, dv = (case[c] for c in ("n", "h", "dk", "dv"))
    l = x["q"].shape[0]
    zero = torch.zeros(n, h, dk, dv, dtype=torch.float64, device="cuda")
    s = zero if leaf["state"] is None else leaf["state"]
    grow = zero
    lengths = torch.full((n,), l, device="cuda") if leaf["lengths"] is None else leaf["lengths"]
    live = (torch.arange(l, device="cuda")[:, None] < lengths)[..., None, None]
    y = torch.zeros(l, n, h, dv, dtype=torch.float64, device="cuda")
    dq = torch.zeros(l, n, h, dk, dtype=torch.float64, device="cuda")
    dg = torch.zeros(h, dtype=torch.float64, device="cuda")
    for t in range(l):
        on = live[t][..., None]
        if kind == "attn_grad" and case["decay"]:
            grow = torch.where(on, decay * (grow + s), grow)
        s = torch.where(on, decay * s + x["k"][t][..., None] * x["v"][t][..., None, :], s)
        if kind != "attn_grad":
            y[t] = torch.where(live[t], torch.matmul(x["q"][t][..., None, :], s)[..., 0, :] * leaf["scale"], 0.0)
            continue
        d = torch.where(live[t], x["dy"][t] * leaf["scale"], 0.0)
        dq[t] = torch.matmul(s, d[..., None])[..., 0]
        if case["decay"]:
            dg += (x["q"][t] * torch.matmul(grow, d[..., None])[..., 0]).sum((0, 2))
    if kind != "attn_grad":
        return (y[0] if one else y.movedim(0, 1)), s
    back = zero if leaf["dstate"] is None else leaf["dstate"]
    dg += (back * grow).sum((0, 2, 3))
    dk_, dv_ = torch.zeros_like(dq), y
    for t in range(l - 1, -1, -1):
        on = live[t][..., None]
        d = x["dy"][t] * leaf["scale"]
        g = back + x["q"][t][..., None] * d[..., None, :]
        dk_[t] = torch.where(live[t], torch.matmul(g, x["v"][t][..., None])[..., 0], 0.0)
        dv_[t] = torch.where(live[t], torch.matmul(x["k"][t][..., None, :], g)[..., 0, :], 0.0)
        back = torch.where(on, decay * g, back)
    out = [t.movedim(0, 1) for t in (dq, dk_, dv_)]
    if case["decay"]:
        out.append(dg)
    return out + ([back] if leaf["state"] is not None else [])
