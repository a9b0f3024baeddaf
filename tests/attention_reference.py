"""Plain 64-bit implementations of the root-mean-square norm, rotary positions and
linear attention, and the magnitudes their error bounds are stated in (the
bounds themselves: seq_reference.check).  They run where their inputs are."""
import torch


def wide(t):
    return None if t is None else t.detach().double()


# ------------------------------------------------------------------ root-mean-square norm

def rms_norm(x, residual, w, eps):
    """y, z, rstd, and the magnitude of y's terms."""
    z = x if residual is None else x + residual
    terms = x.abs() if residual is None else x.abs() + residual.abs()
    rstd = ((z * z).mean(-1, keepdim=True) + eps) ** -0.5
    w1 = torch.ones(x.shape[-1], dtype=torch.float64, device=x.device) if w is None else w
    # an error of z moves rstd by at most its relative size in the row's norm
    near = terms.square().mean(-1, keepdim=True).sqrt() * rstd
    return z * rstd * w1, z, rstd[..., 0], (terms + z.abs() * near) * rstd * w1.abs()


def rms_norm_backward(dy, x, rstd, w, dsum, absolute=False):
    """dx, dw; absolute: with every term taken by its absolute value."""
    r = rstd[..., None]
    xh = x * r
    g = dy if w is None else dy * w
    if absolute:
        xh, g, dy = xh.abs(), g.abs(), dy.abs()
        dx = r * (g + xh * (g * xh).mean(-1, keepdim=True))
        more = None if dsum is None else dsum.abs()
    else:
        dx = r * (g - xh * (g * xh).mean(-1, keepdim=True))
        more = dsum
    return dx if more is None else dx + more, (dy * xh).sum(tuple(range(x.dim() - 1)))


def scales(y, group):
    """max |y| / 448 of each row or group, at least 2^-100."""
    rows = y.unflatten(-1, (-1, group or y.shape[-1]))
    s = (rows.abs().amax(-1) / 448.0).clamp(min=2.0 ** -100)
    return s if group else s[..., 0]


# ------------------------------------------------------------------ rotary positions

def rotary(x, freqs, at, interleaved, scale, sign=1):
    """x [..., H, D] turned, and the magnitude of its terms; at: positions [...]."""
    angle = at.double()[..., None, None] * freqs * sign
    c, s = torch.cos(angle) * scale, torch.sin(angle) * scale
    half = freqs.shape[0]
    if interleaved:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
    else:
        a, b = x[..., :half], x[..., half:2 * half]
    y, mag = x.clone(), torch.zeros_like(x)
    p, q, m = a * c - b * s, a * s + b * c, (a.abs() + b.abs()) * abs(scale)
    if interleaved:
        y[..., 0:2 * half:2], y[..., 1:2 * half:2] = p, q
        mag[..., 0:2 * half:2], mag[..., 1:2 * half:2] = m, m
    else:
        y[..., :half], y[..., half:2 * half] = p, q
        mag[..., :half], mag[..., half:2 * half] = m, m
    return y, mag


# ------------------------------------------------------------------ linear attention

def _live(lengths, n, l, device):
    m = torch.full((n,), l, device=device) if lengths is None else lengths.to(device).long().clamp(0, l)
    return torch.arange(l, device=device)[:, None] < m


def _zeros(n, h, dk, dv, like):
    return torch.zeros(n, h, dk, dv, dtype=torch.float64, device=like.device)


def attention(q, k, v, g, scale, state, lengths):
    """y [N,L,H,DV] and the last state, position by position."""
    n, l, h, dk = q.shape
    s = _zeros(n, h, dk, v.shape[-1], q) if state is None else state
    decay = torch.exp(g)[:, None, None]
    live = _live(lengths, n, l, q.device)
    y = torch.zeros(n, l, h, v.shape[-1], dtype=torch.float64, device=q.device)
    for t in range(l):
        on = live[t][:, None, None, None]
        s = torch.where(on, decay * s + k[:, t, :, :, None] * v[:, t, :, None, :], s)
        y[:, t] = torch.where(on[..., 0], scale * (q[:, t, :, :, None] * s).sum(-2), 0.0)
    return y, s


def attention_backward(dy, q, k, v, g, scale, state, lengths, dlast):
    """dict of the gradients of q, k, v, log_decay and state by the formulas.  With every
    argument taken by its absolute value: the magnitudes of their terms."""
    n, l, h, dk = q.shape
    dv = v.shape[-1]
    s = _zeros(n, h, dk, dv, q) if state is None else state
    grow = torch.zeros_like(s)  # the state's derivative by log_decay
    decay = torch.exp(g)[:, None, None]
    live = _live(lengths, n, l, q.device)
    r = dict(q=torch.zeros_like(q), k=torch.zeros_like(k), v=torch.zeros_like(v),
             log_decay=torch.zeros(h, dtype=torch.float64, device=q.device))
    for t in range(l):
        on = live[t][:, None, None, None]
        grow = torch.where(on, decay * (grow + s), grow)
        s = torch.where(on, decay * s + k[:, t, :, :, None] * v[:, t, :, None, :], s)
        d = torch.where(on[..., 0], scale * dy[:, t], 0.0)
        r["q"][:, t] = (s * d[:, :, None, :]).sum(-1)
        r["log_decay"] += (q[:, t] * (grow * d[:, :, None, :]).sum(-1)).sum((0, 2))
    back = torch.zeros_like(s) if dlast is None else dlast
    r["log_decay"] += (back * grow).sum((0, 2, 3))
    for t in range(l - 1, -1, -1):
        on = live[t][:, None, None, None]
        at = back + scale * q[:, t, :, :, None] * dy[:, t, :, None, :]
        r["k"][:, t] = torch.where(on[..., 0], (at * v[:, t, :, None, :]).sum(-1), 0.0)
        r["v"][:, t] = torch.where(on[..., 0], (at * k[:, t, :, :, None]).sum(-2), 0.0)
        back = torch.where(on, decay * at, back)
    r["state"] = back
    return r


def absolute(*args):
    return [a.abs() if torch.is_tensor(a) and a.is_floating_point() else a for a in args]
