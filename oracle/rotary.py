"""FP64 oracle of the rotary operators (TEST INFRASTRUCTURE ONLY).

Plain numpy in float64 from the closed forms; shares no code with the CUDA
library.  Besides the values it returns, element by element, how far an FP32
evaluation of the same formulas may be from them, and replays the order of the
weight gradients in float32.

Arrays are [tokens, heads, D].  U is the relative rounding error of one FP32
operation.  A cosine or sine of the kernels is off by at most 4 U: the angle by
2 pi (2^-32 + 2^-34) = 0.03 U (top 32 bits of the fraction of a turn; turns per
position rounded to 2^-65, positions below 2^31), the Taylor polynomials by 0.03 U,
their roundings by less than 2 U (sine) and 3 U (cosine); the product with scale
adds one more rounding.
"""
from __future__ import annotations

from fractions import Fraction

import numpy as np

U = 2.0 ** -24
ANGLE = 5               # U of a cosine or sine, times scale
# U of 1 / rms: a sum of squares of depth 16 (4 products and 5 additions of a lane, 5 of a team, 1/D and the
# rounding with eps), halved by the root, and 2.5 of the root (one Newton step: its products and its sum)
RSTD = 12

# 1 / (2 pi) to 400 bits, from Machin's formula in integers
def _inverse_turn(bits: int = 400) -> Fraction:
    one = 1 << (bits + 16)

    def arctan_inverse(n):
        total, power, k = 0, one // n, 0
        while power:
            total += (-1) ** k * (power // (2 * k + 1))
            power //= n * n
            k += 1
        return total

    pi = 4 * (4 * arctan_inverse(5) - arctan_inverse(239))
    return Fraction(one, 2 * pi)


INVERSE_TURN = _inverse_turn()


def turns(frequency: float) -> Fraction:
    """Turns per position of a frequency in radians per position."""
    return Fraction(float(frequency)) * INVERSE_TURN


def cos_sin_far(position: int, frequency: float):
    """Cosine and sine at any position: the fraction of a turn exactly, then float64."""
    t = turns(frequency) * int(position)
    t -= round(t)
    a = 2 * np.pi * float(t)
    return np.cos(a), np.sin(a)


def pairs(rotary_dim: int, first: int, interleaved: bool):
    i = np.arange(rotary_dim // 2)
    return (first + 2 * i, first + 2 * i + 1) if interleaved else (first + i, first + rotary_dim // 2 + i)


def rotate(x, position, freq, rotary_dim, first, interleaved, scale=1.0, back=False):
    """(y, err) of [T, H, D] heads at positions [T] (|position| up to 2^20 or so)."""
    x = np.asarray(x, dtype=np.float64)
    a, b = pairs(rotary_dim, first, interleaved)
    angle = np.asarray(position, dtype=np.float64)[:, None] * np.asarray(freq)[None, :]
    c, s = (scale * np.cos(angle))[:, None], (scale * np.sin(angle))[:, None]
    if back:
        s = -s
    y, err = x.copy(), np.zeros_like(x)
    xa, xb = x[..., a], x[..., b]
    y[..., a], y[..., b] = xa * c - xb * s, xb * c + xa * s
    e = (ANGLE + 2) * U * abs(scale) * (np.abs(xa) + np.abs(xb))
    err[..., a], err[..., b] = e, e
    return y, err


def _spread(v, rotary_dim, first, interleaved, scale):
    """Per element: the sizes that meet in a rotated element (its own column's outside)."""
    a, b = pairs(rotary_dim, first, interleaved)
    out = np.abs(v).copy()
    both = abs(scale) * (np.abs(v[..., a]) + np.abs(v[..., b]))
    out[..., a], out[..., b] = both, both
    return out


def forward(x, w, position, freq, rotary_dim, first, interleaved, scale, eps):
    """(y, err) of norm and rotation: z = x rstd w is off by (RSTD + 2) U of itself."""
    x = np.asarray(x, dtype=np.float64)
    rstd = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    z = x * rstd * w
    y, err = rotate(z, position, freq, rotary_dim, first, interleaved, scale)
    return y, err + (RSTD + 2) * U * _spread(z, rotary_dim, first, interleaved, scale)


def backward(x, w, dy, position, freq, rotary_dim, first, interleaved, scale, eps):
    """(dx, dweight, err_dx, err_dw), dx unrounded.

    g = rot'(dy) as in rotate; a = g w; the row's sum of a x has depth 15; xhat is off by
    (RSTD + 1) U of itself.  The weight gradient adds its terms along chains of 16 heads,
    10 tokens, the chunks (at most as many as heads), the groups of one of 512 shares (of 5 and more tokens,
    or at most 2 x 3648 smaller ones; 64 shares of up to 256 groups), 2 steps between the shares of a
    warp, 16 warps and 8 CTAs."""
    x = np.asarray(x, dtype=np.float64)
    D = x.shape[-1]
    rstd = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    xhat = x * rstd
    g, eg = rotate(dy, position, freq, rotary_dim, first, interleaved, scale, back=True)
    a = g * w
    ea = np.abs(w) * eg + U * np.abs(a)
    m = (a * xhat).mean(-1, keepdims=True)
    em = rstd * ((np.abs(x) * ea).sum(-1, keepdims=True) + 15 * U * np.abs(a * x).sum(-1, keepdims=True)) / D \
        + (RSTD + 3) * U * np.abs(m)                     # its three products and 1/D on top of the root's
    t = a - xhat * m
    dx = rstd * t
    et = ea + np.abs(xhat) * em + (RSTD + 1) * U * np.abs(xhat * m) + U * np.abs(t)
    err = rstd * et + (RSTD + 1) * U * np.abs(dx)
    term = g * xhat
    n = x.shape[0]
    chain = 16 + 10 + x.shape[1] + 1 + max(n // (512 * 5) + 1, 15) + 2 + 24
    err_dw = (np.abs(xhat) * eg).sum((0, 1)) + (RSTD + 2 + chain) * U * np.abs(term).sum((0, 1))
    return dx, term.sum((0, 1)), err, err_dw


def rounded(err, ref, dtype: str):
    """Bound after one rounding to the type: half a step of the value (bf16 2^-8, fp16 2^-11 of it),
    or half the smallest subnormal, on top of the FP32 error."""
    half, tiny = {"bfloat16": (2.0 ** -8, 2.0 ** -134), "float16": (2.0 ** -11, 2.0 ** -25), "float32": (0.0, 0.0)}[dtype]
    return err + half * (np.abs(ref) + err) + tiny


def grad_replay(q_leaf: np.ndarray, k_leaf: np.ndarray):
    """float32 replay of both weight gradients' order for exact leaves g xhat [tokens, heads, D]."""
    n, hq, D = q_leaf.shape
    heads = hq + k_leaf.shape[1]
    leaf = np.concatenate([q_leaf, k_leaf], 1).astype(np.float32)
    lanes = (D + 15) // 16                                            # of a head; teams are of these or the next power of two
    size = 1 << (lanes - 1).bit_length()
    size = lanes if 32 // lanes > 32 // size else size
    teams = 32 // size
    group = 8 if teams > 10 else teams if teams >= 5 else 8 // teams * teams
    while group // 2 >= teams and group > 2 and -(-n // group) * -(-heads // 8) <= 3648:
        group //= 2
    tokens = max(1, group // teams)                                   # of a group, added up by one team
    groups = -(-n // group)
    best = None
    for most in (16, 12, 8, 6, 4, 3, 2):
        c = -(-heads // most)
        time = -(-groups * c // 2432) * (tokens * (-(-heads // c) + 2) + 2)
        if best is None or time < best:
            best, chunks = time, c
    per = (heads + chunks - 1) // chunks
    slots = -(-hq // per) + (chunks - hq // per if heads > hq else 0)
    ctas = 1 if groups <= 256 and slots <= 8 else 8
    shares = ctas * 16 * 4
    share = (groups + shares - 1) // shares
    out = []
    for lo, hi in ((0, hq), (hq, heads)):
        value = []
        for g in range(groups):
            v = None
            for c in range(chunks):
                mine = range(max(lo, c * per), min(hi, c * per + per))
                if not len(mine):
                    continue
                u = None
                for first in range(group * g, min(group * g + group, n), tokens):
                    part = None
                    for t in range(first, min(first + tokens, n)):
                        s = np.zeros(D, np.float32)
                        for h in mine:
                            s = s + leaf[t, h]
                        part = s if part is None else part + s
                    u = part if u is None else u + part
                v = u if v is None else v + u
            value.append(v)
        part = []
        for r in range(shares):
            acc = np.zeros(D, np.float32)
            for g in range(r * share, min((r + 1) * share, groups)):
                acc = acc + value[g]
            part.append(acc)
        w = 16 * ctas
        warps = [(part[i] + part[w + i]) + (part[2 * w + i] + part[3 * w + i]) for i in range(w)]
        total = None
        for r in range(ctas):
            s = warps[16 * r]
            for w in range(1, 16):
                s = s + warps[16 * r + w]
            total = s if total is None else total + s
        out.append(total)
    return out
