"""The operators of a softmax attention layer in 64 bits (angles in the 80 bits
of numpy's long double), from their definitions, and the error bounds of their
kernels.  U and ROUND as in tests/_layer.py."""
from __future__ import annotations

import numpy as np

from tests._layer import ROUND, U

LD = np.longdouble
PI2 = 2 * LD("3.14159265358979323846264338327950288")


def theta(rot, kind="plain", base=10000.0, factor=1.0, orig_len=0.0, lo=1.0, hi=32.0, divisors=None):
    """Angles per position of the pairs, in long double."""
    base = LD(base)
    if kind == "base" and rot > 2:
        base = base * LD(factor) ** (LD(rot) / LD(rot - 2))
    i = np.arange(rot // 2, dtype=LD)
    t = base ** (-2 * i / LD(rot))
    keep = np.ones(rot // 2, dtype=LD)
    if kind == "linear":
        keep = keep * 0
    elif kind == "turns":
        keep = np.clip((LD(orig_len) * t / PI2 - LD(lo)) / (LD(hi) - LD(lo)), 0, 1)
    elif kind == "index":
        at = [LD(rot) / 2 * np.log(LD(orig_len) / (PI2 * LD(n))) / np.log(base) for n in (hi, lo)]
        i0, i1 = max(np.floor(at[0]), LD(0)), min(np.ceil(at[1]), LD(rot - 1))
        if i0 == i1:
            i1 = i1 + LD("0.001")
        keep = 1 - np.clip((i - i0) / (i1 - i0), 0, 1)
    if kind != "base":
        t = keep * t + (1 - keep) * t / LD(factor)
    return t / np.asarray(divisors, dtype=LD) if divisors is not None else t


def rotate(x, pos, th, rot, inter=False, inverse=False, amp=1.0):
    """x [n, heads, d] turned by pos [n], and the bound of the fp32 kernel
    without the output's rounding.

    The angle is exact to 2^-30; cos and sin of it carry three roundings of the
    argument (|y| <= pi/4: 2.4 u) and 2.5 of the series, the factor one: 6 u of
    amp.  Then the two products and their sum round once each: 9 u of
    amp (|a| + |b|) in all, written 10."""
    x = np.asarray(x, np.float64)
    t = (np.asarray(pos).astype(LD)[:, None] * th) % PI2
    c, s = (np.cos(t) * LD(amp)).astype(np.float64)[:, None], (np.sin(t) * LD(amp)).astype(np.float64)[:, None]
    s = -s if inverse else s
    a_at, b_at = (slice(0, rot, 2), slice(1, rot, 2)) if inter else (slice(0, rot // 2), slice(rot // 2, rot))
    y, err = x.copy(), np.zeros(x.shape)
    a, b = x[..., a_at], x[..., b_at]
    y[..., a_at], y[..., b_at] = a * c - b * s, b * c + a * s
    err[..., a_at] = err[..., b_at] = 10 * U * amp * (np.abs(a) + np.abs(b))
    return y, err


def attend(q, K, V, scale):
    """One cache head: q [G, d], K and V [n, d] in 64 bits.  Returns o [G, d],
    the weights [G, n], and the relative error of a weight and the bound of o
    (without the output's rounding).

    A score is a sum of d exact or rounded products in fp32, scaled in a few
    roundings: (d + 8) u sum |q k| scale.  The difference to the running maximum
    rounds relative to itself, exp2 is one ulp, and each of the factors between
    two maxima is one such rounding: (8 + 2 n/16) u and 4 u per unit of the scores' range.
    Two bf16 parts of a weight leave 2^-17 of it.  Sum and output are sums of n
    terms in fp32."""
    n = K.shape[0]
    if n == 0:
        return np.zeros((q.shape[0], V.shape[1])), np.zeros((q.shape[0], 0)), 0.0, 0.0
    s = q @ K.T * scale
    mag = (np.abs(q) @ np.abs(K).T * scale).max()
    w = np.exp(s - s.max(-1, keepdims=True))
    w = w / w.sum(-1, keepdims=True)
    rng = (s.max(-1) - s.min(-1)).max()
    eta = (2 * (q.shape[1] + 8) * mag + 8 + n / 8 + 4 * rng) * U + 2.0 ** -17
    o = w @ V
    return o, w, 2 * eta + n * U, (w @ np.abs(V)) * (2 * eta + 2 * n * U)


def evict(acc, pos, budget, sink, recent):
    """One head of one entry: (holes, rows that move into them) of acc and pos [n]."""
    n = len(acc)
    stay = (pos < sink) | (pos.astype(np.int64) > int(pos.max()) - recent)
    gone = np.zeros(n, bool)
    gone[np.lexsort((np.arange(n), np.where(stay, 0.0, acc), stay))[:n - budget]] = True
    return np.flatnonzero(gone[:budget]), np.flatnonzero(~gone[budget:]) + budget


__all__ = ["LD", "ROUND", "U", "attend", "evict", "rotate", "theta"]
