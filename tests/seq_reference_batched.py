"""The 64-bit references of seq_reference.py for all sequences and positions at
once, on any device: the same formulas with masks in the place of cut sequences,
for sizes that step by step on the CPU would take minutes.  Only the scan's
recurrences run along the positions."""
import torch

from seq_reference import sigmoid, softplus


def _valid(lengths, n, l, device):
    """[n, l] truth values of the valid positions."""
    if lengths is None:
        return torch.ones(n, l, dtype=torch.bool, device=device)
    return torch.arange(l, device=device)[None, :] < lengths.to(device).long()[:, None]


def _cut(t, valid):
    return torch.where(valid[..., None], t, torch.zeros((), dtype=t.dtype, device=t.device))


# ------------------------------------------------------------------ causal convolution

def _rows(x, w, state, lengths):
    n, l, c = x.shape
    k = w.shape[1]
    valid = _valid(lengths, n, l, x.device)
    head = torch.zeros(n, k - 1, c, dtype=torch.float64, device=x.device) if state is None else state
    return torch.cat([head, _cut(x, valid)], 1), valid


def _pre(rows, w, b, l, absolute):
    f = torch.abs if absolute else (lambda t: t)
    pre = torch.zeros_like(rows[:, :l])
    for j in range(w.shape[1]):
        pre = pre + f(rows[:, j:j + l] * w[:, j])
    return pre if b is None else pre + f(b)


def causal_conv(x, w, b, act, state, lengths):
    """y, the last state, and the magnitude of pre's terms."""
    n, l, c = x.shape
    k = w.shape[1]
    rows, valid = _rows(x, w, state, lengths)
    pre = _pre(rows, w, b, l, False)
    at = torch.full((n,), l, device=x.device) if lengths is None else lengths.to(x.device).long().clamp(0, l)
    at = at[:, None] + torch.arange(k - 1, device=x.device)
    last = torch.gather(rows, 1, at[..., None].expand(n, k - 1, c))
    return (_cut(pre * sigmoid(pre) if act else pre, valid), last, _cut(_pre(rows, w, b, l, True), valid))


def causal_conv_backward(dy, x, w, b, act, state, lengths, dlast, absolute=False):
    """dx, dw, db, dstate; absolute: the magnitudes of their terms."""
    n, l, c = x.shape
    k = w.shape[1]
    rows, valid = _rows(x, w, state, lengths)
    d = _cut(dy, valid)
    if act:
        pre = _pre(rows, w, b, l, False)
        s = sigmoid(pre)
        d = d.abs() * (1.1 + 0.5 * _pre(rows, w, b, l, True)) if absolute else d * s * (1 + pre * (1 - s))
    elif absolute:
        d = d.abs()
    f = torch.abs if absolute else (lambda t: t)
    d = _cut(d, valid)
    drows = torch.zeros_like(rows)
    if dlast is not None:
        at = torch.full((n,), l, device=x.device) if lengths is None else lengths.to(x.device).long().clamp(0, l)
        at = at[:, None] + torch.arange(k - 1, device=x.device)
        drows.scatter_(1, at[..., None].expand(n, k - 1, c), f(dlast))
    dw = torch.empty_like(w)
    for j in range(k):
        drows[:, j:j + l] += d * f(w[:, j])
        dw[:, j] = (d * f(rows[:, j:j + l])).sum((0, 1))
    return _cut(drows[:, k - 1:], valid), dw, d.sum((0, 1)), drows[:, :k - 1]


# ------------------------------------------------------------------ selective scan

def _first(t):
    return t.transpose(0, 1).contiguous()


def scan(u, delta, a, b, c, skip, gate, bias, plus, state, lengths, absolute=False, keep=None):
    """y and the last state; absolute: with every term taken by its absolute value.
    keep: a dict that takes position-first tensors."""
    n, l, d = u.shape
    f = torch.abs if absolute else (lambda t: t)
    valid = _valid(lengths, n, l, u.device)
    raw = delta if bias is None else delta + bias
    u, step, b, c = (_first(_cut(t, valid)) for t in (u, softplus(raw) if plus else raw, b, c))
    decay = torch.exp(step[..., None] * a)
    h = torch.empty(l + 1, *decay.shape[1:], dtype=torch.float64, device=u.device)
    h[1:] = f((step * u)[..., None] * b[:, :, None, :])
    h[0] = 0.0 if state is None else f(state)
    for t in range(l):
        h[t + 1].addcmul_(decay[t], h[t])
    y = (h[1:] * f(c)[:, :, None, :]).sum(-1)
    if skip is not None:
        y = y + f(skip * u)
    if keep is not None:
        keep.update(u=u, step=step, b=b, c=c, raw=_first(raw), decay=decay, h=h, y=y, valid=valid)
    if gate is not None:
        z = _first(_cut(gate, valid))
        y = y * f(z * sigmoid(z))
    return _cut(y.transpose(0, 1), valid), h[l].clone()


def scan_backward(dy, u, delta, a, b, c, skip, gate, bias, plus, state, lengths, dlast, absolute=False):
    """(u, delta, a, b, c, skip, gate, bias, state) gradients by the formula;
    absolute: the magnitudes of their terms."""
    f = torch.abs if absolute else (lambda t: t)
    k = {}
    scan(u, delta, a, b, c, skip, gate, bias, plus, state, lengths, absolute=absolute, keep=k)
    valid, u, step, b, c, decay, h = (k[x] for x in ("valid", "u", "step", "b", "c", "decay", "h"))
    l = u.shape[0]
    back = lambda t: t.transpose(0, 1).contiguous()
    g, r = _first(_cut(dy, valid)), {}
    if gate is not None:
        z = _first(_cut(gate, valid))
        s = sigmoid(z)
        r["gate"] = back(g.abs() * k["y"] * (1.1 + 0.5 * z.abs()) if absolute else g * k["y"] * s * (1 + z * (1 - s)))
        g = g * z * s
    g = f(g)
    gh = g[..., None] * f(c)[:, :, None, :]
    if dlast is not None:
        gh[l - 1] += f(dlast)
    for t in range(l - 2, -1, -1):
        gh[t].addcmul_(decay[t + 1], gh[t + 1])
    gb = (gh * f(b)[:, :, None, :]).sum(-1)
    r["u"] = back(f(step) * gb + (0 if skip is None else f(skip) * g))
    r["b"] = back((gh * f(step * u)[..., None]).sum(2))
    r["c"] = back((h[1:] * g[..., None]).sum(2))
    r["skip"] = (g * f(u)).sum((0, 1))
    gh *= decay
    r["state"] = gh[0].clone()
    gh *= h[:-1]
    draw = (gh * f(a)).sum(-1) + f(u) * gb
    if plus:
        draw = draw * sigmoid(k["raw"])
    r["delta"] = _cut(back(draw), valid)
    r["bias"] = r["delta"].sum((0, 1))
    r["a"] = (gh * f(step)[..., None]).sum((0, 1))
    return r
