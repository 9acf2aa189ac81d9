"""The operators around a recurrent state in 64 bits, from their definitions
and token by token, and the error bounds of their kernels.

Bounds count roundings: u = 2^-24 is fp32's half step relative to a value
(bf16: 2^-8 of it, written ROUND).  A sum of n terms formed in fp32 in any
order is off by at most n u sum|terms|.  The hardware exp2, reciprocal and
reciprocal square root are within one ulp (2 u)."""
from __future__ import annotations

import numpy as np

U = 2.0 ** -24
ROUND = {"bf16": 2.0 ** -8, "f32": U}


def sigmoid(x):
    return 0.5 * (1.0 + np.tanh(0.5 * x))


def softplus(v):
    return np.maximum(v, 0.0) + np.log1p(np.exp(-np.abs(v)))


def silu_bound(a, err):
    """Error of a * sigmoid(a) in fp32 for an argument off by err: silu' lies
    in (-0.1, 1.1); e^-a carries its argument's rounding (|a| u, twice) and
    exp2's ulp, then 1 + e, the reciprocal and the product round."""
    return 1.1 * err + np.abs(a * sigmoid(a)) * (2 * np.abs(a) + 8) * U


def conv_rows(x, hist, w, bias, silu):
    """y [n,C], the new history, and the bound without the output's rounding,
    for one sequence x [n,C] after hist [W-1,C]."""
    W, n = w.shape[0], x.shape[0]
    e = np.concatenate([hist, x])
    b = np.zeros(x.shape[1]) if bias is None else bias
    a = b + sum(w[k] * e[k:k + n] for k in range(W))
    mag = np.abs(b) + sum(np.abs(w[k] * e[k:k + n]) for k in range(W))
    err = W * U * mag
    if silu:
        return a * sigmoid(a), e[n:], silu_bound(a, err)
    return a, e[n:], err


def ssm_rows(x, B, C, dt, A, D, dt_bias, S, *, sp=True, lo=0.0, hi=np.inf):
    """One sequence token by token: x [n,H,dv], B and C [n,H,dk] (repeated to
    the heads), dt [n,H], S [H,dk,dv] (not changed).  Returns y, the state,
    the same two of magnitudes (every product by its absolute value), the
    step sizes and the arguments of their softplus."""
    n, H, dv = x.shape
    S, Sm = S.astype(np.float64).copy(), np.abs(S.astype(np.float64))
    v = dt + (0.0 if dt_bias is None else dt_bias)
    delta = np.clip(softplus(v) if sp else v, lo, hi)
    y, ym = np.empty((n, H, dv)), np.empty((n, H, dv))
    for t in range(n):
        a = np.exp(delta[t] * A)[:, None, None]
        S = a * S + B[t][:, :, None] * (delta[t][:, None] * x[t])[:, None, :]
        Sm = a * Sm + np.abs(B[t])[:, :, None] * np.abs(delta[t][:, None] * x[t])[:, None, :]
        y[t] = np.matmul(C[t][:, None, :], S)[:, 0]
        ym[t] = np.matmul(np.abs(C[t])[:, None, :], Sm)[:, 0]
        if D is not None:
            y[t] += D[:, None] * x[t]
            ym[t] += np.abs(D[:, None] * x[t])
    return y, S, ym, Sm, delta, v


def delta_bound(v):
    """Relative error of delta: the sum's rounding moves softplus by at most
    |v| u of itself (softplus' <= softplus), e^v and log1p add a few ulps."""
    return (np.abs(v) + 10) * U


def rms_rows(u, eps):
    return 1.0 / np.sqrt((u * u).mean(-1, keepdims=True) + eps)
