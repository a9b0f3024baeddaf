"""Measured cases of the sequence operators: layer norm, the short causal
convolution and the selective state space scan, each forward, backward and (the
convolution and the scan) for single tokens.

``run`` has two forms.  With ``own`` false it computes the operator from its
formula with elementary torch operations in 32 bits, rounded once at the end;
with ``own`` true it calls the package.  ``exact`` computes the same outputs in
64 bits, apart from both: the backward passes there are automatic
differentiation of the 64-bit forward definition, the scan there is computed by
recursive doubling instead of step by step.

Formulas (n: sequence, t: position, c or d: channel, s: state):

  layer norm          y = (x - mean) * rstd * w + b,  rstd = 1 / sqrt(var + eps)
  causal convolution  y[t,c] = act(b[c] + sum_k w[c,k] * X[t+k,c]),  X = K-1 rows of
                      state followed by x; the new state is the last K-1 valid rows
  scan                D = softplus(delta + delta_bias)
                      h[t,d,s] = exp(D[t,d] a[d,s]) h[t-1,d,s] + D[t,d] u[t,d] b[t,s]
                      y[t,d] = (sum_s c[t,s] h[t,d,s] + skip[d] u[t,d]) * silu(gate[t,d])

``lengths`` gives each sequence's valid positions; past them outputs and
gradients are 0 and the state stands still.
"""
import math

import torch

own = False

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
EPS = 1e-5

# ------------------------------------------------------------------ cases


def listed():
    return [
        # one token's activations between the layers of a model that is answering
        {"name": "norm-one-token", "kind": "norm", "dtype": "bf16", "n": 1, "l": 1, "c": 512},
        # rows of an odd count and a width that fills no power of two, before a half-precision layer
        {"name": "norm-odd", "kind": "norm", "dtype": "f16", "n": 1, "l": 3001, "c": 1000},
        # a training step's activations of wide rows
        {"name": "norm-wide", "kind": "norm", "dtype": "bf16", "n": 8, "l": 4096, "c": 4096},
        # the same in the backward direction, rows as wide as the scan's channels
        {"name": "norm-grad", "kind": "norm_grad", "dtype": "bf16", "n": 8, "l": 2048, "c": 2048},
        # the pixels of a batch of 56 x 56 images with 512 channels, in 32 bits
        {"name": "norm-grad-image", "kind": "norm_grad", "dtype": "f32", "n": 8, "l": 3136, "c": 512},
        # prompts through the convolution; the input is one half of a wider projection's rows
        {"name": "conv-prompt", "kind": "conv", "dtype": "bf16", "n": 4, "l": 4096, "c": 4096, "k": 4, "split": True,
         "ragged": False, "state": True},
        # training on sequences of several lengths
        {"name": "conv-grad-ragged", "kind": "conv_grad", "dtype": "f16", "n": 5, "l": 2047, "c": 2048, "k": 4,
         "split": False, "ragged": True, "state": False},
        # one new token of each of 64 sequences
        {"name": "conv-token", "kind": "conv_step", "dtype": "bf16", "n": 64, "c": 4096, "k": 4},
        # one long prompt
        {"name": "scan-long", "kind": "scan", "dtype": "bf16", "n": 1, "l": 16384, "d": 2048, "s": 16, "split": True,
         "ragged": False, "state": False},
        # a batch of prompts of several lengths that go on from their states, an odd width, in 32 bits
        {"name": "scan-ragged", "kind": "scan", "dtype": "f32", "n": 6, "l": 1023, "d": 1000, "s": 16, "split": False,
         "ragged": True, "state": True},
        # a training step
        {"name": "scan-grad", "kind": "scan_grad", "dtype": "bf16", "n": 8, "l": 2048, "d": 2048, "s": 16,
         "split": True, "ragged": False, "state": False},
        # one new token of each of 64 sequences
        {"name": "scan-token", "kind": "scan_step", "dtype": "f16", "n": 64, "d": 4096, "s": 16},
    ]


def _log(rng, lo, hi):
    """An integer of [lo, hi], spread over the logarithm, odd and even ones alike."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    kind = rng.choice(["norm", "norm_grad", "conv", "conv_grad", "conv_step", "scan", "scan", "scan_grad",
                       "scan_step"])
    case = {"kind": kind, "dtype": rng.choice(["f32", "f16", "bf16"])}
    if kind in ("norm", "norm_grad"):
        c = _log(rng, 32, 8192)
        n = _log(rng, 1, 8)
        l = _log(rng, 1, max(1, min(8192, (1 << 26) // (c * n))))
        return {**case, "n": n, "l": l, "c": c}
    if kind == "conv_step":
        return {**case, "n": _log(rng, 1, 128), "c": _log(rng, 64, 8192), "k": rng.choice([2, 3, 4, 4])}
    if kind == "scan_step":
        return {**case, "n": _log(rng, 1, 128), "d": _log(rng, 64, 8192), "s": rng.choice([8, 16, 16, 32, 64])}
    flags = {"split": rng.random() < 0.5, "ragged": rng.random() < 0.5, "state": rng.random() < 0.5}
    n = _log(rng, 1, 8)
    if kind in ("conv", "conv_grad"):
        c = _log(rng, 64, 8192)
        l = _log(rng, 1, max(1, min(8192, (1 << 25) // (c * n))))
        return {**case, "n": n, "l": l, "c": c, "k": rng.choice([2, 3, 4, 4]), **flags}
    d, s = _log(rng, 64, 4096), rng.choice([8, 16, 16, 32, 64])
    l = _log(rng, 1, max(1, min(4096, (1 << 27) // (d * n * s))))
    return {**case, "n": n, "l": l, "d": d, "s": s, **flags}


def work(case):
    e = SIZE[case["dtype"]]
    kind = case["kind"]
    if kind in ("norm", "norm_grad"):
        rows, c = case["n"] * case["l"], case["c"]
        if kind == "norm":  # x, w, b read; y, mean and rstd written
            return {"bytes": e * (2 * rows * c + 2 * c) + 8 * rows, "flops": 8 * rows * c}
        return {"bytes": e * (3 * rows * c + 3 * c) + 8 * rows, "flops": 14 * rows * c}
    if kind == "conv_step":
        n, c, k = case["n"], case["c"], case["k"]
        return {"bytes": e * (2 * n * c + 2 * n * (k - 1) * c + c * (k + 1)), "flops": (2 * k + 5) * n * c}
    if kind == "scan_step":
        n, d, s = case["n"], case["d"], case["s"]
        return {"bytes": 8 * n * d * s + 4 * d * s + 8 * d + e * (4 * n * d + 2 * n * s), "flops": 7 * n * d * s}
    n, l = case["n"], case["l"]
    live = sum(_lengths(case)) if case["ragged"] else n * l
    if kind in ("conv", "conv_grad"):
        c, k = case["c"], case["k"]
        state = e * n * (k - 1) * c
        if kind == "conv":
            return {"bytes": e * (live * c + n * l * c + c * (k + 1)) + (2 if case["state"] else 1) * state,
                    "flops": (2 * k + 5) * live * c}
        return {"bytes": e * (2 * live * c + n * l * c + 2 * c * (k + 1)) + (2 * state if case["state"] else 0),
                "flops": (6 * k + 9) * live * c}
    d, s = case["d"], case["s"]
    state, params = 4 * n * d * s, 4 * (d * s + 2 * d)
    if kind == "scan":  # u, delta, gate, b, c read, y written
        return {"bytes": e * (live * (3 * d + 2 * s) + n * l * d) + params + (2 if case["state"] else 1) * state,
                "flops": 7 * live * d * s}
    return {"bytes": e * (live * (4 * d + 2 * s) + n * l * (3 * d + 2 * s)) + 2 * params
            + (2 * state if case["state"] else 0), "flops": 20 * live * d * s}


# ------------------------------------------------------------------ inputs


def _lengths(case):
    """Valid positions: one full sequence, one of a single token, one of none, the rest between."""
    n, l = case["n"], case["l"]
    fixed = [l, 1, 0]
    return [fixed[i] if i < 3 else 1 + (i * 7919 + l // 2) % l for i in range(n)]


def _inputs(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1000003 + 17)
    dt = DT[case["dtype"]]
    kind = case["kind"]

    def normal(*shape, scale=1.0, shift=0.0, dtype=dt):
        return (torch.randn(shape, generator=g, device="cuda") * scale + shift).to(dtype)

    def uniform(*shape, lo=0.0, hi=1.0):
        return torch.rand(shape, generator=g, device="cuda") * (hi - lo) + lo

    if kind in ("norm", "norm_grad"):
        n, l, c = case["n"], case["l"], case["c"]
        st = {"x": normal(n, l, c, scale=1.5, shift=0.25), "w": normal(c, scale=0.1, shift=1.0),
              "b": normal(c, scale=0.1)}
        if kind == "norm_grad":
            st["dy"] = normal(n, l, c)
            xf = st["x"].float()  # the statistics that the forward pass left
            mean = xf.mean(-1)
            st["mean"] = mean
            st["rstd"] = ((xf - mean[..., None]).square().mean(-1) + EPS).rsqrt()
        return st
    if kind == "conv_step":
        n, c, k = case["n"], case["c"], case["k"]
        st = {"x": normal(n, c), "state": normal(n, k - 1, c), "w": normal(c, k, scale=k ** -0.5),
              "b": normal(c, scale=0.1)}
        st["new_state"] = torch.empty_like(st["state"])
        return st
    if kind == "scan_step":
        n, d, s = case["n"], case["d"], case["s"]
        st = _scan_params(d, s, normal, uniform)
        st.update(u=normal(n, d), delta=normal(n, d, scale=0.5), gate=normal(n, d), b=normal(n, s), c=normal(n, s),
                  state=normal(n, d, s, scale=0.1, dtype=torch.float32))
        st["new_state"] = torch.empty_like(st["state"])
        return st
    n, l = case["n"], case["l"]
    st = {"lengths": None, "state": None}
    if case["ragged"]:
        st["lengths"] = torch.tensor(_lengths(case), dtype=torch.int32, device="cuda")
    if kind in ("conv", "conv_grad"):
        c, k = case["c"], case["k"]
        st["x"] = normal(n, l, 2 * c)[..., :c] if case["split"] else normal(n, l, c)
        st["w"] = normal(c, k, scale=k ** -0.5)
        st["b"] = normal(c, scale=0.1)
        if case["state"]:
            st["state"] = normal(n, k - 1, c)
        if kind == "conv_grad":
            st["dy"] = normal(n, l, c)
        return st
    d, s = case["d"], case["s"]
    st.update(_scan_params(d, s, normal, uniform))
    if case["split"]:  # u and gate, b and c as parts of wider projections' rows
        ug, bc = normal(n, l, 2 * d), normal(n, l, 2 * s + 64)
        st.update(u=ug[..., :d], gate=ug[..., d:], b=bc[..., 64:64 + s], c=bc[..., 64 + s:])
    else:
        st.update(u=normal(n, l, d), gate=normal(n, l, d), b=normal(n, l, s), c=normal(n, l, s))
    st["delta"] = normal(n, l, d, scale=0.5)
    if case["state"]:
        st["state"] = normal(n, d, s, scale=0.1, dtype=torch.float32)
    if kind == "scan_grad":
        st["dy"] = normal(n, l, d)
    return st


def _scan_params(d, s, normal, uniform):
    """Decays of 1 to s per unit of time, steps of 0.001 to 0.1 units where delta is 0."""
    step = torch.exp(uniform(d, lo=math.log(1e-3), hi=math.log(1e-1)))
    a = -torch.arange(1, s + 1, device="cuda", dtype=torch.float32).repeat(d, 1) * uniform(d, s, lo=0.9, hi=1.1)
    return {"a": a, "skip": normal(d, scale=0.1, shift=1.0, dtype=torch.float32),
            "delta_bias": step + torch.log(-torch.expm1(-step))}


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
    if kind == "norm":
        return cn.layer_norm(st["x"], st["w"], st["b"], EPS, return_stats=True)
    if kind == "norm_grad":
        return cn.layer_norm_backward(st["dy"], st["x"], st["mean"], st["rstd"], st["w"])
    if kind == "conv":
        return cn.causal_conv1d(st["x"], st["w"], st["b"], activation="silu", state=st["state"],
                                lengths=st["lengths"], return_state=True)
    if kind == "conv_grad":
        r = cn.causal_conv1d_backward(st["dy"], st["x"], st["w"], st["b"], activation="silu", state=st["state"],
                                      lengths=st["lengths"])
        return [t for t in (r.x, r.w, r.bias, r.state) if t is not None]
    if kind == "conv_step":
        y = cn.causal_conv1d_step(st["x"], st["state"], st["w"], st["b"], activation="silu",
                                  state_out=st["new_state"])
        return y, st["new_state"]
    if kind == "scan":
        return cn.selective_scan(st["u"], st["delta"], st["a"], st["b"], st["c"], skip=st["skip"], gate=st["gate"],
                                 delta_bias=st["delta_bias"], softplus=True, state=st["state"],
                                 lengths=st["lengths"], return_state=True)
    if kind == "scan_grad":
        r = cn.selective_scan_backward(st["dy"], st["u"], st["delta"], st["a"], st["b"], st["c"], skip=st["skip"],
                                       gate=st["gate"], delta_bias=st["delta_bias"], softplus=True,
                                       state=st["state"], lengths=st["lengths"])
        return [t for t in (r.u, r.delta, r.a, r.b, r.c, r.skip, r.gate, r.delta_bias, r.state) if t is not None]
    y = cn.selective_scan_step(st["u"], st["delta"], st["a"], st["b"], st["c"], st["state"], skip=st["skip"],
                               gate=st["gate"], delta_bias=st["delta_bias"], softplus=True,
                               state_out=st["new_state"])
    return y, st["new_state"]


def _run_plain(st):
    kind = st["kind"]
    if kind == "norm":
        return _plain_norm(st)
    if kind == "norm_grad":
        return _plain_norm_grad(st)
    if kind == "conv":
        return _plain_conv(st)
    if kind == "conv_grad":
        return _plain_conv_grad(st)
    if kind == "conv_step":
        x = st["x"].float()
        rows = torch.cat([st["state"].float(), x[:, None]], 1)
        pre = (rows * st["w"].float().t()).sum(1) + st["b"].float()
        st["new_state"].copy_(rows[:, 1:])
        return (pre * _sigmoid(pre)).to(st["x"].dtype), st["new_state"]
    if kind == "scan":
        return _plain_scan(st)
    if kind == "scan_grad":
        return _plain_scan_grad(st)
    u = st["u"].float()
    step = _softplus(st["delta"].float() + st["delta_bias"])
    h = torch.exp(step[..., None] * st["a"]) * st["state"] + (step * u)[..., None] * st["b"].float()[:, None, :]
    st["new_state"].copy_(h)
    y = (h * st["c"].float()[:, None, :]).sum(-1) + st["skip"] * u
    z = st["gate"].float()
    return (y * z * _sigmoid(z)).to(st["u"].dtype), st["new_state"]


def _sigmoid(x):
    return 1.0 / (1.0 + torch.exp(-x))


def _softplus(x):
    return torch.clamp(x, min=0.0) + torch.log1p(torch.exp(-x.abs()))


def _valid(st, l):
    """[n, l, 1] truth values of the valid positions, or None."""
    if st["lengths"] is None:
        return None
    return (torch.arange(l, device="cuda")[None, :] < st["lengths"][:, None])[..., None]


def _masked(t, valid):
    return t if valid is None else torch.where(valid, t, torch.zeros((), dtype=t.dtype, device=t.device))


def _plain_norm(st):
    x = st["x"].float()
    mean = x.mean(-1, keepdim=True)
    xc = x - mean
    rstd = 1.0 / torch.sqrt((xc * xc).mean(-1, keepdim=True) + EPS)
    y = xc * rstd * st["w"].float() + st["b"].float()
    return y.to(st["x"].dtype), mean[..., 0], rstd[..., 0]


def _plain_norm_grad(st):
    x, dy, rstd = st["x"].float(), st["dy"].float(), st["rstd"][..., None]
    xh = (x - st["mean"][..., None]) * rstd
    g = dy * st["w"].float()
    dx = rstd * (g - g.mean(-1, keepdim=True) - xh * (g * xh).mean(-1, keepdim=True))
    return dx.to(st["x"].dtype), (dy * xh).sum((0, 1)).to(st["w"].dtype), dy.sum((0, 1)).to(st["w"].dtype)


def _rows(st):
    """K-1 rows of state, then x with its positions past the lengths cleared."""
    x = st["x"].float()
    n, l, c = x.shape
    k = st["w"].shape[1]
    head = torch.zeros(n, k - 1, c, device="cuda") if st["state"] is None else st["state"].float()
    return torch.cat([head, _masked(x, _valid(st, l))], 1)


def _plain_conv(st):
    rows, w = _rows(st), st["w"].float()
    n, l, c = st["x"].shape
    k = w.shape[1]
    pre = st["b"].float() + sum(rows[:, j:j + l] * w[:, j] for j in range(k))
    y = _masked(pre * _sigmoid(pre), _valid(st, l)).to(st["x"].dtype)
    if st["lengths"] is None:
        return y, rows[:, l:].to(st["x"].dtype)
    at = st["lengths"].long()[:, None] + torch.arange(k - 1, device="cuda")
    return y, torch.gather(rows, 1, at[..., None].expand(n, k - 1, c)).to(st["x"].dtype)


def _plain_conv_grad(st):
    rows, w, dt = _rows(st), st["w"].float(), st["x"].dtype
    n, l, c = st["x"].shape
    k = w.shape[1]
    valid = _valid(st, l)
    pre = st["b"].float() + sum(rows[:, j:j + l] * w[:, j] for j in range(k))
    sig = _sigmoid(pre)
    dpre = _masked(st["dy"].float() * sig * (1.0 + pre * (1.0 - sig)), valid)
    drows = torch.zeros_like(rows)
    dw = torch.empty(c, k, device="cuda")
    for j in range(k):
        drows[:, j:j + l] += dpre * w[:, j]
        dw[:, j] = (dpre * rows[:, j:j + l]).sum((0, 1))
    out = [_masked(drows[:, k - 1:], valid).to(dt), dw.to(dt), dpre.sum((0, 1)).to(dt)]
    if st["state"] is not None:
        out.append(drows[:, :k - 1].to(dt))
    return out


def _scan_terms(st):
    """Position-first tensors of the recurrence; positions past the lengths leave the state as it is."""
    u, raw = st["u"].float(), st["delta"].float() + st["delta_bias"]
    b, c = st["b"].float(), st["c"].float()
    valid = _valid(st, u.shape[1])
    u, step, b, c = (_masked(t, valid) for t in (u, _softplus(raw), b, c))
    first = [t.transpose(0, 1).contiguous() for t in (u, step, b, c)]
    return first, raw.transpose(0, 1), valid


def _plain_states(u, step, a, b, state):
    """decay [l,n,d,s] and h with one more position in front: h[t+1] = decay[t] h[t] + step u b."""
    l, n, d = u.shape
    decay = torch.exp(step[..., None] * a)
    h = torch.empty(l + 1, n, d, a.shape[1], device="cuda")
    torch.mul((step * u)[..., None], b[:, :, None, :], out=h[1:])
    h[0] = 0.0 if state is None else state
    for t in range(l):
        h[t + 1].addcmul_(decay[t], h[t])
    return decay, h


def _plain_scan(st):
    (u, step, b, c), _, valid = _scan_terms(st)
    _, h = _plain_states(u, step, st["a"], b, st["state"])
    y = (h[1:] * c[:, :, None, :]).sum(-1) + st["skip"] * u
    z = st["gate"].float()
    y = _masked(y.transpose(0, 1) * z * _sigmoid(z), valid)
    return y.to(st["u"].dtype).contiguous(), h[-1].clone()


def _plain_scan_grad(st):
    (u, step, b, c), raw, valid = _scan_terms(st)
    a, dt = st["a"], st["u"].dtype
    l = u.shape[0]
    decay, h = _plain_states(u, step, a, b, st["state"])
    z = st["gate"].float().transpose(0, 1)
    dy = st["dy"].float()
    dy = _masked(dy, valid).transpose(0, 1)
    sig = _sigmoid(z)
    y = (h[1:] * c[:, :, None, :]).sum(-1) + st["skip"] * u
    dgate = dy * y * sig * (1.0 + z * (1.0 - sig))
    dy = dy * z * sig
    g = dy[..., None] * c[:, :, None, :]
    for t in range(l - 2, -1, -1):
        g[t].addcmul_(decay[t + 1], g[t + 1])
    gb = (g * b[:, :, None, :]).sum(-1)
    du = step * gb + st["skip"] * dy
    kept = g * decay
    dstate = kept[0].clone()
    kept *= h[:-1]  # g * (what the decay multiplies, decayed)
    dstep = (kept * a).sum(-1) + u * gb
    ddelta = dstep * _sigmoid(raw)
    if valid is not None:
        ddelta = _masked(ddelta, valid.transpose(0, 1))
    da = (kept * step[..., None]).sum((0, 1))
    db = (g * (step * u)[..., None]).sum(2)
    dc = (h[1:] * dy[..., None]).sum(2)

    def back(t):
        return t.transpose(0, 1).to(dt).contiguous()

    out = [back(du), back(ddelta), da, back(db), back(dc), (dy * u).sum((0, 1)), back(dgate), ddelta.sum((0, 1))]
    if st["state"] is not None:
        out.append(dstate)
    return out


# ------------------------------------------------------------------ 64 bits


def exact(case, seed):
    st = _inputs(case, seed)
    kind = case["kind"]
    leaf = {k: v.double() if torch.is_tensor(v) and v.is_floating_point() else v for k, v in st.items()}
    del st
    if kind == "norm":
        x = leaf["x"]
        var, mean = torch.var_mean(x, -1, unbiased=False)
        rstd = (var + EPS) ** -0.5
        return (x - mean[..., None]) * rstd[..., None] * leaf["w"] + leaf["b"], mean, rstd
    if kind == "norm_grad":
        # the statistics are the forward pass's, so they are functions of x here
        x, w = leaf["x"].requires_grad_(), leaf["w"].requires_grad_()
        b = torch.zeros_like(leaf["w"]).requires_grad_()
        var, mean = torch.var_mean(x, -1, unbiased=False, keepdim=True)
        y = (x - mean) * (var + EPS) ** -0.5 * w + b
        return torch.autograd.grad(y, (x, w, b), leaf["dy"])
    if kind == "conv_step":
        rows = torch.cat([leaf["state"], leaf["x"][:, None]], 1)
        pre = torch.matmul(rows.permute(2, 0, 1).contiguous(), leaf["w"][:, :, None]).squeeze(-1).t() + leaf["b"]
        return pre / (1 + torch.exp(-pre)), rows[:, 1:]
    if kind in ("conv", "conv_grad"):
        return _exact_conv(leaf, kind == "conv_grad")
    if kind == "scan_step":
        step = torch.logaddexp(leaf["delta"] + leaf["delta_bias"], torch.zeros((), dtype=torch.float64, device="cuda"))
        h = leaf["state"] * torch.exp(step[:, :, None] * leaf["a"]) + torch.matmul(
            (step * leaf["u"])[:, :, None], leaf["b"][:, None, :])
        y = torch.matmul(h, leaf["c"][:, :, None]).squeeze(-1) + leaf["skip"] * leaf["u"]
        z = leaf["gate"]
        return y * z / (1 + torch.exp(-z)), h
    return _exact_scan(leaf, kind == "scan_grad")


def _exact_conv(leaf, grad):
    """Sequence by sequence, each cut to its own length."""
    x, w, b, state = leaf["x"], leaf["w"], leaf["b"], leaf["state"]
    n, l, c = x.shape
    k = w.shape[1]
    lengths = [l] * n if leaf["lengths"] is None else leaf["lengths"].tolist()
    y, last = torch.zeros(n, l, c, dtype=torch.float64, device="cuda"), []
    dx, dstate = torch.zeros_like(y), torch.zeros(n, k - 1, c, dtype=torch.float64, device="cuda")
    dw, db = torch.zeros_like(w), torch.zeros_like(b)
    for i, m in enumerate(lengths):
        head = torch.zeros(k - 1, c, dtype=torch.float64, device="cuda") if state is None else state[i]
        rows = torch.cat([head, x[i, :m]], 0)
        last.append(rows[m:].clone())
        if m == 0:
            continue
        leaves = [t.detach().clone().requires_grad_(grad) for t in (rows, w, b)]
        windows = leaves[0].unfold(0, k, 1)  # [m, c, k]
        pre = (windows * leaves[1]).sum(-1) + leaves[2]
        out = pre / (1 + torch.exp(-pre))
        if not grad:
            y[i, :m] = out
            continue
        dr, dwi, dbi = torch.autograd.grad(out, leaves, leaf["dy"][i, :m])
        dx[i, :m], dstate[i] = dr[k - 1:], dr[:k - 1]
        dw += dwi
        db += dbi
    if not grad:
        return y, torch.stack(last)
    return [dx, dw, db] + ([dstate] if state is not None else [])


def _doubled(decay, h):
    """All states of h[t] = decay[t] h[t-1] + h[t] along dimension 1, by recursive doubling."""
    reach = 1
    while reach < h.shape[1]:
        h = torch.cat([h[:, :reach], h[:, reach:] + decay[:, reach:] * h[:, :-reach]], 1)
        decay = torch.cat([decay[:, :reach], decay[:, reach:] * decay[:, :-reach]], 1)
        reach *= 2
    return h


def _exact_scan(leaf, grad):
    """Sequence by sequence, each cut to its own length, some channels at a time."""
    names = ["u", "delta", "a", "b", "c", "skip", "gate", "delta_bias"]
    n, l, d = leaf["u"].shape
    s = leaf["a"].shape[1]
    lengths = [l] * n if leaf["lengths"] is None else leaf["lengths"].tolist()
    y = torch.zeros(n, l, d, dtype=torch.float64, device="cuda")
    start = torch.zeros(n, d, s, dtype=torch.float64, device="cuda") if leaf["state"] is None else leaf["state"]
    final = start.clone()
    grads = {k: torch.zeros(leaf[k].shape, dtype=torch.float64, device="cuda") for k in names}
    dstate = torch.zeros_like(start)
    for i, m in enumerate(lengths):
        if m == 0:
            continue
        wide = max(1, min(d, (1 << (25 if grad else 28)) // (m * s)))
        for d0 in range(0, d, wide):
            cut = slice(d0, min(d, d0 + wide))
            at = {"u": (i, slice(0, m), cut), "delta": (i, slice(0, m), cut), "a": (cut,), "b": (i, slice(0, m)),
                  "c": (i, slice(0, m)), "skip": (cut,), "gate": (i, slice(0, m), cut), "delta_bias": (cut,)}
            v = {k: leaf[k][at[k]].detach().clone().requires_grad_(grad) for k in names}
            h0 = start[i, cut].detach().clone().requires_grad_(grad)
            step = torch.logaddexp(v["delta"] + v["delta_bias"],
                                   torch.zeros((), dtype=torch.float64, device="cuda")).t()  # [d, m]
            decay = torch.exp(step[:, :, None] * v["a"][:, None, :])
            push = (step * v["u"].t())[:, :, None] * v["b"]
            h = _doubled(decay, torch.cat([push[:, :1] + decay[:, :1] * h0[:, None], push[:, 1:]], 1))
            out = (h * v["c"]).sum(-1).t() + v["skip"] * v["u"]
            out = out * v["gate"] / (1 + torch.exp(-v["gate"]))
            if not grad:
                y[i, :m, cut], final[i, cut] = out, h[:, -1]
                continue
            got = torch.autograd.grad(out, [v[k] for k in names] + [h0], leaf["dy"][i, :m, cut])
            for k, t in zip(names, got):
                grads[k][at[k]] += t
            dstate[i, cut] = got[-1]
    if not grad:
        return y, final
    out = [grads[k] for k in names]
    return out + ([dstate] if leaf["state"] is not None else [])
