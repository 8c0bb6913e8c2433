"""Norms and rotation of queries and keys, and their gradients, in 64 bits, with bounds on what a
computation in 32 bits may be off by."""
from __future__ import annotations

import math

import torch

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
TINY = {"bf16": 2.0 ** -134, "f16": 2.0 ** -25}  # half the least step


def out_round(dtype):
    """What a value may be off by, relative, when it is rounded once."""
    return torch.finfo(TYPES[dtype]).eps / 2


def frequencies(rot, base=10000.0):
    return [base ** (-2.0 * f / rot) for f in range(rot // 2)]


def angles(positions, freq, axes=None):
    """[tokens, rot / 2] radians in 64 bits; positions [tokens] or [axes, tokens] int32."""
    pos = positions.double()
    f = torch.tensor(freq, dtype=torch.float64, device=pos.device)
    if axes is None:
        return pos.reshape(-1)[:, None] * f
    return torch.stack([pos[a].reshape(-1) * f[i] for i, a in enumerate(axes)], -1)


def turn(x, angle, interleaved, back=False):
    """x [tokens, heads, d] with its first channels rotated by `angle` [tokens, rot / 2]."""
    if angle is None:
        return x.clone()
    half = angle.shape[-1]
    c, s = torch.cos(angle)[:, None], torch.sin(angle)[:, None]
    s = -s if back else s
    a = (slice(0, 2 * half, 2) if interleaved else slice(0, half))
    b = (slice(1, 2 * half, 2) if interleaved else slice(half, 2 * half))
    y = x.clone()
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def partner(x, angle, interleaved):
    """Magnitudes |x_a| + |x_b| of each channel's pair (|x| outside the pairs)."""
    y = x.abs().clone()
    if angle is None:
        return y
    half = angle.shape[-1]
    a = (slice(0, 2 * half, 2) if interleaved else slice(0, half))
    b = (slice(1, 2 * half, 2) if interleaved else slice(half, 2 * half))
    both = y[..., a] + y[..., b]
    y[..., a], y[..., b] = both, both
    return y


def forward(x, weight, angle, interleaved, norm, eps):
    """(y, bound in 32 bits) of one side, x [tokens, heads, d].

    With u = 2^-24: the sum of d squares (positive terms, in a tree and chains of 8) is off by 16 u at
    most relative, its mean by 1 more, rsqrtf by 4 u (two ulps), so r by (17 / 2 + 4) u < 13 u; the two
    products by r and w add 2 u.  A cosine or sine (sincospif's error 2^-23 at most, its argument's
    rounding pi 2^-25, a turn's lower bits left out 2 pi 2^-32, the reference's angle in 64 bits below
    2^-26 for positions to 2^27) is off by 4 u absolute, the rotation's products and sum add 2 u.  In all
    (15 + 4 + 2) u < 24 u of |n_a| + |n_b|."""
    x = x.double()
    n = x
    if norm:
        n = x / torch.sqrt(x.square().mean(-1, keepdim=True) + eps)
        if weight is not None:
            n = n * weight.double()
    return turn(n, angle, interleaved), 24 * 2.0 ** -24 * partner(n, angle, interleaved)


def backward(x, dy, weight, angle, interleaved, norm, eps):
    """(dx, its bound, dw, its bound) of one side.

    dn is off by 6 u of its pair's magnitudes (above).  xh = x r by 14 u, g = dn w by 7 u of its pair;
    the mean of g xh by (14 + 7 + 12) u of the mean of |g| |xh| (d products and sums in chains of 8 and a
    tree), dx = r (g - xh m) by 13 u + 3 u more: 64 u of r (|g| + |xh| mean(|g| |xh|)) with |g| for the
    pair covers all.  dw: each term 21 u of |dn| |xh|, sums in chains of at most 2^12 terms (a thread's
    rows) and 64 (a CTA's groups), then in 64 bits: at most 2^12 u + 85 u more, were all roundings one
    way.  Roundings of sums do not all go one way: an independent rounding error of u / 2 of the partial
    sum each, and partial sums no larger than the sum of magnitudes of the chain so far, give a standard
    deviation below u sqrt(chain) times the chain's sum of magnitudes; 8 of those and the terms' own 21 u
    are allowed."""
    x, dy, d = x.double(), dy.double(), x.shape[-1]
    dn = turn(dy, angle, interleaved, back=True)
    size = partner(dy, angle, interleaved)
    u = 2.0 ** -24
    if not norm:
        return dn, 6 * u * size, None, None
    r = 1 / torch.sqrt(x.square().mean(-1, keepdim=True) + eps)
    xh = x * r
    w = weight.double() if weight is not None else torch.ones(d, dtype=torch.float64, device=x.device)
    g, gs = dn * w, size * w.abs()
    dx = r * (g - xh * (g * xh).mean(-1, keepdim=True))
    bound = 64 * u * r * (gs + xh.abs() * (gs * xh.abs()).mean(-1, keepdim=True))
    terms = (size * xh.abs()).flatten(0, 1).sum(0)
    return dx, bound, (dn * xh).flatten(0, 1).sum(0), (21 + 8 * math.sqrt(2 ** 12)) * u * terms


def check(name, got, want, bound, dtype):
    """`got` rounds something within `bound` of `want` once; a NaN fails."""
    want = want.reshape(got.shape)
    bound = bound.reshape(got.shape)
    if dtype is not None:
        bound = bound + out_round(dtype) * (want.abs() + bound) + TINY[dtype]
    err = (got.double() - want).abs()
    assert (err <= bound).all(), (name, int((~(err <= bound)).sum()), float((err / bound.clamp(min=1e-300)).max()))


def exact_angles(positions, freq):
    """angles() for positions as far as an int32 goes, by whole numbers."""
    from fractions import Fraction
    two_pi = Fraction(2 * 3141592653589793238462643383279502884197169399375105820974945, 10 ** 60)
    rows = [[float(Fraction(f) * p % two_pi) for f in freq] for p in positions]
    return torch.tensor(rows, dtype=torch.float64)
