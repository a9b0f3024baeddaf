"""How far a 16-bit linear attention may be from the 64-bit one in the norm: the bound
that an error of a few percent does not pass, where the bound of each element, which
counts every term by its absolute value, would let it.

y, dq, dk and dv are rounded once, and so is an operand of each of the two products that
they are sums of; a rounding is off by u at most and, over many values, by u / sqrt(6) or
so of their norm.  Values of random signs keep that through a sum: sqrt(2) u / sqrt(6)
= 0.58 u for both (the two products are two parts of one sum).  2 u is 3.4 times as much.
fp32, and the states in every type: each of 32 chunks or runs adds a rounding and its decay's
error of two units, a chunk's products 256 more of random signs: below 2^-19.
"""
import torch

BOUND = {torch.float32: 2.0 ** -19, torch.float16: 2.0 ** -10, torch.bfloat16: 2.0 ** -7}


def far(got, ref, dims):
    """The norm of the difference over the reference's, over dims."""
    g = got.double()
    return (g - ref).square().sum(dims).sqrt() / ref.square().sum(dims).sqrt()


def check(got, ref, dims, where, bound=None):
    d = far(got, ref, dims)
    assert bool((d <= (BOUND[got.dtype] if bound is None else bound)).all()), f"{where}: {d.max().item()} of the norm"
