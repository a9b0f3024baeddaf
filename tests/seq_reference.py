"""Plain 64-bit implementations of the sequence operators, step by step on the
CPU, and the magnitudes their error bounds are stated in.

Every bound is  u |ref| + k * 2^-24 * mag : u the unit roundoff of the output's
type (one rounding at the end), k the number of 32-bit roundings that can add
up, mag the same formula with every term taken by its absolute value.
"""
import numpy as np
import torch

EPS = 2.0 ** -24
ROUND = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 2.0 ** -126, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -126}


def f64(t):
    return None if t is None else t.detach().cpu().double()


def check(got, ref, mag, k, where):
    """|got - ref| <= u |ref| + k 2^-24 mag, element by element (16-bit types' subnormals aside)."""
    g = f64(got)
    assert g.shape == ref.shape, f"{where}: shape {tuple(g.shape)} for {tuple(ref.shape)}"
    assert torch.isfinite(g).all(), f"{where}: non-finite values"
    tol = ROUND[got.dtype] * ref.abs() * (1 + 2 * k * EPS) + k * EPS * mag + TINY[got.dtype]
    bad = (g - ref).abs() > tol
    if bad.any():
        i = tuple(torch.nonzero(bad)[0].tolist())
        raise AssertionError(f"{where}: {int(bad.sum())} of {bad.numel()} out of bound; first at {i}: "
                             f"got {g[i].item()!r}, reference {ref[i].item()!r}, bound {tol[i].item()!r}")


def sigmoid(x):
    return 1.0 / (1.0 + torch.exp(-x))


def softplus(x):
    return torch.clamp(x, min=0) + torch.log1p(torch.exp(-x.abs()))


# ------------------------------------------------------------------ layer norm

def layer_norm(x, w, b, eps):
    """y, mean, rstd and the magnitude of y's terms."""
    mean = x.mean(-1, keepdim=True)
    xc = x - mean
    rstd = 1.0 / torch.sqrt((xc * xc).mean(-1, keepdim=True) + eps)
    xh = xc * rstd
    w1 = torch.ones(x.shape[-1], dtype=torch.float64) if w is None else w
    b0 = torch.zeros(x.shape[-1], dtype=torch.float64) if b is None else b
    mag = (xh.abs() + (x.abs().mean(-1, keepdim=True) + x.abs()) * rstd) * w1.abs() + b0.abs()
    return xh * w1 + b0, mean[..., 0], rstd[..., 0], mag


def layer_norm_backward(dy, x, mean, rstd, w, absolute=False):
    """dx, dw, db; absolute: with every term taken by its absolute value."""
    r = rstd[..., None]
    xh = (x - mean[..., None]) * r
    g = dy if w is None else dy * w
    if absolute:
        xh, g, dy = xh.abs() + (x.abs() + mean.abs()[..., None]) * r, g.abs(), dy.abs()
        dx = r * (g + g.mean(-1, keepdim=True) + xh * (g * xh).mean(-1, keepdim=True))
    else:
        dx = r * (g - g.mean(-1, keepdim=True) - xh * (g * xh).mean(-1, keepdim=True))
    lead = tuple(range(x.dim() - 1))
    return dx, (dy * xh).sum(lead), dy.sum(lead)


# ------------------------------------------------------------------ causal convolution

def _lengths(lengths, n, l):
    return [l] * n if lengths is None else [min(max(int(v), 0), l) for v in lengths.tolist()]


def causal_conv(x, w, b, act, state, lengths):
    """y, the last state, and the magnitude of pre's terms."""
    n, l, c = x.shape
    k = w.shape[1]
    y, mag = torch.zeros_like(x), torch.zeros_like(x)
    last = torch.zeros(n, k - 1, c, dtype=torch.float64)
    for i, m in enumerate(_lengths(lengths, n, l)):
        head = torch.zeros(k - 1, c, dtype=torch.float64) if state is None else state[i]
        rows = torch.cat([head, x[i, :m]], 0)
        for t in range(m):
            pre, a = torch.zeros(c, dtype=torch.float64), torch.zeros(c, dtype=torch.float64)
            for j in range(k):
                pre = pre + w[:, j] * rows[t + j]
                a = a + (w[:, j] * rows[t + j]).abs()
            if b is not None:
                pre, a = pre + b, a + b.abs()
            y[i, t] = pre * sigmoid(pre) if act else pre
            mag[i, t] = a
        last[i] = rows[m:]
    return y, last, mag


def causal_conv_backward(dy, x, w, b, act, state, lengths, dlast, absolute=False):
    """dx, dw, db, dstate; absolute: the magnitudes of their terms (with what an
    error of pre does to act')."""
    n, l, c = x.shape
    k = w.shape[1]
    dx, dw, db = torch.zeros_like(x), torch.zeros_like(w), torch.zeros(c, dtype=torch.float64)
    dstate = torch.zeros(n, k - 1, c, dtype=torch.float64)
    wa = w.abs() if absolute else w
    for i, m in enumerate(_lengths(lengths, n, l)):
        head = torch.zeros(k - 1, c, dtype=torch.float64) if state is None else state[i]
        rows = torch.cat([head, x[i, :m]], 0)
        drows = torch.zeros_like(rows)
        if dlast is not None:
            drows[m:] += dlast[i].abs() if absolute else dlast[i]
        for t in range(m):
            pre, a = torch.zeros(c, dtype=torch.float64), torch.zeros(c, dtype=torch.float64)
            for j in range(k):
                pre = pre + w[:, j] * rows[t + j]
                a = a + (w[:, j] * rows[t + j]).abs()
            if b is not None:
                pre, a = pre + b, a + b.abs()
            d = dy[i, t]
            if act:
                s = sigmoid(pre)
                slope = s * (1 + pre * (1 - s))
                d = d.abs() * (1.1 + 0.5 * a) if absolute else d * slope
            elif absolute:
                d = d.abs()
            for j in range(k):
                drows[t + j] += d * wa[:, j]
                dw[:, j] += d * (rows[t + j].abs() if absolute else rows[t + j])
            db += d
        dstate[i], dx[i, :m] = drows[:k - 1], drows[k - 1:]
    return dx, dw, db, dstate


# ------------------------------------------------------------------ selective scan

def scan(u, delta, a, b, c, skip, gate, bias, plus, state, lengths, absolute=False, keep=None):
    """y and the last state; absolute: with every term taken by its absolute value.
    keep: a list that takes (step, decay, states) of every sequence."""
    n, l, d = u.shape
    s = a.shape[1]
    y = torch.zeros_like(u)
    last = torch.zeros(n, d, s, dtype=torch.float64) if state is None else state.clone()
    if absolute:
        last = last.abs()
    for i, m in enumerate(_lengths(lengths, n, l)):
        raw = delta[i, :m] + (0 if bias is None else bias)
        step = softplus(raw) if plus else raw
        h, hs, es = last[i].clone(), [last[i].clone()], []
        for t in range(m):
            e = torch.exp(step[t][:, None] * a)
            push = (step[t] * u[i, t])[:, None] * b[i, t][None, :]
            out = c[i, t][None, :]
            if absolute:
                push, out = push.abs(), out.abs()
            h = e * h + push
            v = (out * h).sum(-1)
            if skip is not None:
                v = v + ((skip * u[i, t]).abs() if absolute else skip * u[i, t])
            if gate is not None:
                z = gate[i, t] * sigmoid(gate[i, t])
                v = v * (z.abs() if absolute else z)
            y[i, t] = v
            hs.append(h)
            es.append(e)
        last[i] = h
        if keep is not None:
            keep.append((raw, step, es, hs))
    return y, last


def scan_backward(dy, u, delta, a, b, c, skip, gate, bias, plus, state, lengths, dlast, absolute=False):
    """(u, delta, a, b, c, skip, gate, delta_bias, state) gradients by the formula;
    absolute: the magnitudes of their terms."""
    n, l, d = u.shape
    s = a.shape[1]
    ab = (lambda t: t.abs()) if absolute else (lambda t: t)
    keep = []
    scan(u, delta, a, b, c, skip, gate, bias, plus, state, lengths, absolute=absolute, keep=keep)
    z = torch.zeros
    r = dict(u=z(n, l, d), delta=z(n, l, d), a=z(d, s), b=z(n, l, s), c=z(n, l, s), skip=z(d), gate=z(n, l, d),
             bias=z(d), state=z(n, d, s))
    r = {k: v.double() for k, v in r.items()}
    for i, m in enumerate(_lengths(lengths, n, l)):
        raw, step, es, hs = keep[i]
        carry = z(d, s).double() if dlast is None else ab(dlast[i]).clone()
        for t in range(m - 1, -1, -1):
            h = hs[t + 1]
            g = dy[i, t]
            if gate is not None:
                zt = gate[i, t]
                sg = sigmoid(zt)
                y = (ab(c[i, t])[None, :] * h).sum(-1)
                if skip is not None:
                    y = y + ab(skip * u[i, t])
                r["gate"][i, t] = g.abs() * y * (1.1 + 0.5 * zt.abs()) if absolute else g * y * sg * (1 + zt * (1 - sg))
                g = g * zt * sg
            g = ab(g)
            gh = g[:, None] * ab(c[i, t])[None, :] + carry
            gb = (gh * ab(b[i, t])[None, :]).sum(-1)
            w = gh * es[t] * hs[t]
            r["u"][i, t] = ab(step[t]) * gb + (0 if skip is None else ab(skip) * g)
            dstep = (w * ab(a)).sum(-1) + ab(u[i, t]) * gb
            draw = dstep * sigmoid(raw[t]) if plus else dstep
            r["delta"][i, t] = draw
            r["bias"] += draw
            r["a"] += w * ab(step[t])[:, None]
            r["b"][i, t] = (gh * ab(step[t] * u[i, t])[:, None]).sum(0)
            r["c"][i, t] = (g[:, None] * h).sum(0)
            r["skip"] += g * ab(u[i, t])
            carry = es[t] * gh
        r["state"][i] = carry
    return r


def directional(f, inputs, name, dots, step=1e-5, seed=0):
    """d/dv of sum(out * dots) along a random v of inputs[name], by central differences, and v."""
    g = torch.Generator().manual_seed(seed)
    v = torch.randn(inputs[name].shape, generator=g, dtype=torch.float64)

    def at(x):
        out = f(**{**inputs, name: inputs[name] + x * v})
        return sum((o * w).sum() for o, w in zip(out, dots) if w is not None)
    return float((at(step) - at(-step)) / (2 * step)), v


def rand(gen, *shape, scale=1.0, shift=0.0):
    return torch.from_numpy(gen.standard_normal(shape, dtype=np.float32)) * scale + shift
