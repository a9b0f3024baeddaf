"""Linear attention in several runs of chunks against the 64-bit reference: every form of a
state (2, 4, 8 and 16 tiles of rows; one and two parts of columns; four and eight wavefronts),
both joins, lengths that end on, before and behind the bounds of runs, rows off 16 bytes,
the longest measured prompt.  Inputs that all three types hold exactly, so that
one reference serves them.

Element by element with the bound of test_gpu_linear_attention.py, and in the norm of
each sequence and head with that of attention_norms.py."""
import functools

import numpy as np
import pytest
import torch

import attention_norms as N
import attention_reference as A
import seq_reference as R

pytestmark = pytest.mark.gpu

cn = pytest.importorskip("convolution_nhwc_conv2d_amd")

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
OPERAND = {"f32": 0, "f16": 1 << 13, "bf16": 1 << 16}
LENGTH = 640


def _shared(g, *shape):
    """Normal values in 8 bits, none of them below 2^-10: exact in float32, float16 and bfloat16."""
    x = R.rand(g, *shape).bfloat16().float()
    return torch.where(x.abs() < 2.0 ** -10, torch.zeros(()), x).cuda()


def _tiles(dk, dv):
    """Rows and columns that a state in lane order has."""
    rows = 32 if dk <= 32 else 64 if dk <= 64 else 128 if dk <= 128 else 256
    return rows, 64 if dv <= 64 else 128 * ((dv + 127) // 128)


def _runs(n, l, h, dk, dv, dt, backward=False):
    """Runs of a pass, from the bytes of the states between them; of a backward pass, whose
    states may be of two forms, whether there are more than one in each."""
    q, v = torch.empty(n, l, h, dk, dtype=DT[dt]), torch.empty(n, l, h, dv, dtype=DT[dt])
    need = cn.linear_attention_workspace_bytes(q, v, backward=backward)
    rows, cols = _tiles(dk, dv)
    if not backward:
        assert need % (n * h * rows * cols * 4) == 0
        return 1 + need // (n * h * rows * cols * 4)
    rows_t, cols_t = _tiles(dv, dk)
    more = cn.linear_attention_workspace_bytes(q, v, backward=True, decay_grad=True) - need
    return need >= n * h * 4 * (rows * cols + 2 * rows_t * cols_t) and more >= n * h * 8 * dk * dv


@functools.lru_cache(maxsize=2)
def _case(n, l, h, dk, dv, lengths, big):
    g = np.random.default_rng([n, l, h, dk, dv])
    i = dict(q=_shared(g, n, l, h, dk), k=_shared(g, n, l, h, dk), v=_shared(g, n, l, h, dv), dy=_shared(g, n, l, h, dv),
             state=_shared(g, n, h, dk, dv) * big, dstate=_shared(g, n, h, dk, dv))
    decay = np.exp(g.uniform(np.log(2e-4), np.log(0.3), h)).astype(np.float32)
    if big > 1:
        decay[:] = np.log(2.0) / 4096
    i["log_decay"] = -torch.from_numpy(decay).cuda()
    m = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
    a = [A.wide(i[x]) for x in ("q", "k", "v", "log_decay")] + [dk ** -0.5, A.wide(i["state"]), m]
    mag = A.absolute(*a)
    mag[3] = a[3]
    dy, ds = A.wide(i["dy"]), A.wide(i["dstate"])
    back, size = A.attention_backward(dy, *a, ds), A.attention_backward(dy.abs(), *mag, ds.abs())
    for r, (y, s) in ((back, A.attention(*a)), (size, A.attention(*mag))):
        r["y"], r["last"] = y, s
    return i, m, back, size


def _placed(t, dt, place):
    """t in its type: dense, or behind `place` elements in rows that are 12 elements longer."""
    t = t.to(DT[dt])
    if not place:
        return t
    n, l, h, d = t.shape
    buf = torch.full((n, l, h * d + 12), float("nan"), dtype=t.dtype, device="cuda")
    view = buf[..., place:place + h * d].unflatten(-1, (h, d))
    view.copy_(t)
    return view


def _elements(got, ref, mag, k, where):
    """seq_reference.check, where the tensors are."""
    g = got.double()
    assert g.shape == ref.shape and bool(torch.isfinite(g).all()), where
    tol = R.ROUND[got.dtype] * ref.abs() * (1 + 2 * k * R.EPS) + k * R.EPS * mag + R.TINY[got.dtype]
    bad = (g - ref).abs() > tol
    assert not bad.any(), f"{where}: {int(bad.sum())} of {bad.numel()} out of bound, first at {torch.nonzero(bad)[0].tolist()}"


def _compare(n, l, h, dk, dv, dt, lengths=None, big=1.0, place=0):
    i, m, want, size = _case(n, l, h, dk, dv, lengths, big)
    q, k, v, dy = (_placed(i[x], dt, place) for x in ("q", "k", "v", "dy"))
    y, last = cn.linear_attention(q, k, v, i["log_decay"], scale=dk ** -0.5, state=i["state"], lengths=m,
                                  return_state=True)
    r = cn.linear_attention_backward(dy, q, k, v, i["log_decay"], scale=dk ** -0.5, state=i["state"], lengths=m,
                                     dstate=i["dstate"], decay_grad=True)
    units = 2 * l + 512
    for name, got in dict(y=y, last=last, **r._asdict()).items():
        what = f"{dk}x{dv} {dt} {name}"
        more = n * l if name == "log_decay" else OPERAND[dt] if name in ("y", "q", "k", "v") else 0
        _elements(got, want[name], size[name], units + more, what)
        if name == "log_decay":
            continue
        full = torch.tensor([x >= 90 for x in lengths]) if lengths else torch.ones(n, dtype=torch.bool)
        dims = (1, 3) if got.dim() == 4 and name not in ("last", "state") else (2, 3)
        N.check(got[full.cuda()], want[name][full.cuda()], dims, what)
        if lengths and dims == (1, 3):
            for x, j in zip(lengths, range(n)):
                assert not got[j, x:].any(), what


SHAPES = [(32, 40), (64, 48), (64, 96), (100, 72), (128, 128), (128, 200), (250, 130), (256, 256)]


@pytest.mark.parametrize("dk,dv", SHAPES)
@pytest.mark.parametrize("dt", list(DT))
def test_runs(dk, dv, dt):
    n, h = 1, 2
    assert _runs(n, LENGTH, h, dk, dv, dt) > 1 and _runs(n, LENGTH, h, dk, dv, dt, backward=True)
    _compare(n, LENGTH, h, dk, dv, dt)


def _heads(dk, dv):
    return 4 if dv <= 128 else 2


def _lengths(dk, dv):
    """None, all, and about the bounds of the runs that the types have, of two to five chunks."""
    at = sorted({32 * -(-(LENGTH // 32) // _runs(8, LENGTH, _heads(dk, dv), dk, dv, dt)) for dt in DT})
    out = [LENGTH, 0, at[0], at[0] + 1, at[-1] - 1, 3 * at[-1], 3 * at[-1] + 17, LENGTH - 1]
    return tuple(min(x, LENGTH) for x in out)


@pytest.mark.parametrize("dk,dv", SHAPES)
@pytest.mark.parametrize("dt", list(DT))
def test_runs_of_ragged_sequences(dk, dv, dt):
    assert _runs(8, LENGTH, _heads(dk, dv), dk, dv, dt) > 1 and _runs(8, LENGTH, _heads(dk, dv), dk, dv, dt, backward=True)
    _compare(8, LENGTH, _heads(dk, dv), dk, dv, dt, lengths=_lengths(dk, dv))


@pytest.mark.parametrize("dk,dv", [(64, 96), (128, 200)])
@pytest.mark.parametrize("dt", list(DT))
def test_runs_that_the_first_state_rules(dk, dv, dt):
    """A state of 30 times the inputs, half of it left after 4096 positions: y is what goes from
    run to run."""
    _compare(1, LENGTH, 2, dk, dv, dt, big=30.0)


@pytest.mark.parametrize("dk,dv", [(64, 96), (100, 72), (250, 130)])
@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("place", [4, 5])
def test_runs_of_rows_off_16_bytes(dk, dv, dt, place):
    _compare(1, LENGTH, 2, dk, dv, dt, place=place)


@pytest.mark.parametrize("n,l,h,dk,dv", [(1, 160, 4, 128, 128), (2, 130, 8, 64, 96)])
@pytest.mark.parametrize("dt", list(DT))
def test_short_sequences_in_runs(n, l, h, dk, dv, dt):
    """As many chunks as fp32 takes in runs, and one more."""
    if dt == "f32":
        assert _runs(n, l, h, dk, dv, dt) > 1
    _compare(n, l, h, dk, dv, dt)


@functools.lru_cache(maxsize=1)
def _long():
    g = np.random.default_rng(7)
    q, k, v = (_shared(g, 1, 16384, 16, 128) for _ in range(3))
    decay = -torch.from_numpy(np.log(2.0) / np.geomspace(4, 4096, 16)).float().cuda()
    return q, k, v, decay, A.attention(A.wide(q), A.wide(k), A.wide(v), A.wide(decay), 128 ** -0.5, None, None)


@pytest.mark.parametrize("dt", list(DT))
def test_a_long_prompt(dt):
    """1 x 16384 x 16 x 128 x 128, half-lives from 4 to 4096: 512 chunks, so 512 roundings of a
    state where the bound of the norm counts 32: of random signs, 4 times as far."""
    assert _runs(1, 16384, 16, 128, 128, dt) > 8
    q, k, v, decay, (ry, rl) = _long()
    y, last = cn.linear_attention(q.to(DT[dt]), k.to(DT[dt]), v.to(DT[dt]), decay, scale=128 ** -0.5, return_state=True)
    more = 4 * N.BOUND[torch.float32]
    N.check(y, ry, (1, 3), "y", max(more, N.BOUND[DT[dt]]))
    N.check(last, rl, (2, 3), "state", more)
