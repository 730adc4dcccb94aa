"""Tight error bounds of the training operations, from the longest chains of additions that the
kernels have (tests/train_reference.py holds the values, and bounds that leave more room).

u = 2^-24.  A sum over a row: a thread adds its slots in two chains of at most 16 pairs (the
kernel for any width: n / 512 elements), one addition joins them, one adds the single element at
a row's end; then 5 levels over a warp, at most 8 additions over the warps of a CTA and 5 levels
over a cluster: at most 40 + n / 512 additions on the way of any term.

A sum over rows: the rows of one thread (rows over the partial rows, of which there are 8 or
more where there are as many rows), the up to 128 rows that share a CTA, a warp's share of the
at most 1216 partial rows (16 warps or more), its 32 warps: at most 240 + rows / 8.
"""
import numpy as np

from train_reference import U


def chain(n):
    return 40 + n / 512


def row_chain(rows):
    return 240 + rows / 8


def layernorm(x, gamma, beta, eps):
    """((y, mean, rstd), their bounds).  The mean is off by dm, the sum's c roundings and the
    quotient's; that shifts every deviation alike, and the mean of their squares by dm^2 at
    most."""
    n = x.shape[1]
    c = chain(n)
    mean = x.mean(1, keepdims=True)
    d = x - mean
    var = (d * d).mean(1, keepdims=True)
    rstd = 1.0 / np.sqrt(var + eps)
    h = d * rstd
    y = h * gamma + beta
    dm = 1.01 * U * (c + 1) * np.abs(x).mean(1, keepdims=True)
    # the squares' mean is off by c + 5 roundings (the deviations' two among them), its sum with
    # eps by one
    rel = (U * (c + 5) * (var + dm * dm) + dm * dm) / (var + eps) + U
    assert (rel < 0.3).all()          # below which the root's second order is less than rel / 2
    rel = 0.5 * rel * (1 + rel) + 5 * U      # rsqrt: two steps
    tol = 1.01 * np.abs(gamma) * (rstd * dm + np.abs(h) * (rel + 2 * U))
    tol = tol + U * (np.abs(y) + tol)
    return (y, mean[:, 0], rstd[:, 0]), (tol, dm[:, 0], (rstd * rel)[:, 0])
