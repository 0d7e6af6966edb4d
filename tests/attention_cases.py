"""Shared by the linear-attention and softmax-attention GPU tests: seeded inputs
on the device with the fp64 values the kernels see, and the error bounds.

Bounds are per element, from the roundings the kernels make.  u = eps / 2 is the
largest relative error of one rounding to the input type, f = 2^-24 of one to
fp32.  bf16 outputs are rounded once (u |o|), and on the way every term of the
sum that forms them at most once (u times the sum of the terms' sizes: the
oracle's bound).  Sums of n fp32 terms are off by at most n f times the sum of
the sizes; powers of the decay and exponentials by a few f each.
"""
import numpy as np
import torch

U = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
F = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def randn(gen, *shape, io="f32", scale=1.0):
    """(device tensor, fp64 host array of exactly its values)."""
    t = (torch.randn(*shape, generator=gen) * scale).to(DT[io])
    return t.cuda(), t.double().numpy()


def fused(gen, lead, widths, io, scales):
    """Tensors [*lead, heads, dim] that are slices of one projection, and their values."""
    x = torch.cat([torch.randn(*lead, h * d, generator=gen) * s for (h, d), s in zip(widths, scales)],
                  dim=-1).to(DT[io])
    out, at, g = [], 0, x.cuda()
    for h, d in widths:
        out.append((g[..., at:at + h * d].unflatten(-1, (h, d)),
                    x[..., at:at + h * d].unflatten(-1, (h, d)).double().numpy()))
        at += h * d
    return out


def host(t):
    return t.detach().double().cpu().numpy()


def within(got, want, bound, what):
    """|got - want| <= bound everywhere (and finite)."""
    got = host(got) if isinstance(got, torch.Tensor) else got
    assert got.shape == want.shape, (what, got.shape, want.shape)
    assert np.isfinite(got).all(), f"{what}: non-finite values"
    bad = np.abs(got - want) > bound
    if bad.any():
        at = np.unravel_index(np.argmax(np.abs(got - want) - bound), want.shape)
        raise AssertionError(f"{what}: {bad.sum()} of {bad.size} values out of bounds, worst at {at}: "
                             f"{got[at]} for {want[at]}, bound {np.broadcast_to(bound, want.shape)[at]:.3g}")


def lin_bounds(io, o, ao, A, L, dk):
    """Bounds of (o, state) of a linear-attention call over L tokens.  fp32 sums
    run over at most L + dk terms, and each term carries a few factors (the power
    of the decay, the weight, the epochs' rescales: 16 roundings to be safe)."""
    n = (L + dk + 16) * F
    bo = n * ao + (U[io] * (np.abs(o) + (1 + U[io]) * ao) if io == "bf16" else F * np.abs(o))
    return bo + 1e-30, n * A + 1e-30


def attn_bound(io, o, ao, big, lk, D):
    """Bound of a softmax-attention output.  A score is a sum of D products
    (relative to their sizes, (D + 3) f), so a probability and the sum it is
    divided by are each off by that times the largest score (and a few f for the
    exponential); the sums over keys by (lk + 8) f; in bf16 each probability is
    rounded once and the output once."""
    eps = 2 * ((D + 3) * F * big + 8 * F) + 2 * (lk + 8) * F
    b = 1.01 * eps * ao + F * np.abs(o)
    if io == "bf16":
        b = b + U[io] * (np.abs(o) + 1.01 * ao)
    return b + 1e-30
