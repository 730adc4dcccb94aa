"""Tight error bounds of the training operations, from the longest chains of additions that the
kernels have (tests/train_reference.py holds the values, and bounds that leave more room).

u = 2^-24.  A sum over a row: a thread adds its slots in two chains of at most 16 pairs (the
kernel for any width: n / 512 elements), one addition joins them, one adds the single element at
a row's end; then 5 levels over a warp, at most 8 additions over the warps of a CTA and 5 levels
over a cluster: at most 40 + n / 512 additions on the way of any term.

A sum over rows: the rows of one thread (of rows over eight clusters or more, or over more
CTAs), the up to 128 rows that share a CTA, a warp's share of the at most 608 partial rows (four
for each of 152 SMs, over 16 warps or more), then up to 32 warps: 1 + rows / 8 + 128 + 38 + 32,
at most 240 + rows / 8.
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


def layernorm_backward(dy, x, gamma, mean, rstd, dstream=None):
    """((dx, dgamma, dbeta), their bounds), from the forward's f32 mean and rstd.  xh carries two
    roundings, w one, a sum c and a product's three, the means' factors three more: c + 12 in
    all of what dx adds up; xh and its product three in a sum over rows."""
    rows, n = x.shape
    rstd = rstd[:, None]
    return _backward(dy, (x - mean[:, None]) * rstd, gamma, rstd, dstream, chain(n) + 12,
                     row_chain(rows) + 4, row_chain(rows), True)


def rmsnorm_backward(dy, x, gamma, eps, dstream=None):
    """((dx, dgamma), their bounds).  inv carries half of its sum's c + 3 roundings and rsqrt's
    two steps, c / 2 + 6; what dx adds up has it three times, beside a sum and seven products."""
    rows, n = x.shape
    c = chain(n)
    inv = 1.0 / np.sqrt((x * x).mean(1, keepdims=True) + eps)
    (dx, dg, _), (tdx, tdg, _) = _backward(dy, x * inv, gamma, inv, dstream, 2.5 * c + 28,
                                           row_chain(rows) + c / 2 + 10, 0, False)
    return (dx, dg), (tdx, tdg)


def _backward(dy, xh, gamma, rstd, dstream, roundings, gamma_roundings, beta_roundings, centred):
    w = dy * gamma
    c1 = w.mean(1, keepdims=True) if centred else np.zeros_like(rstd)
    c2 = (w * xh).mean(1, keepdims=True)
    ds = rstd * (w - c1 - xh * c2)
    parts = np.abs(w) + np.abs(w).mean(1, keepdims=True) * centred \
        + np.abs(xh) * np.abs(w * xh).mean(1, keepdims=True)
    tol = 1.01 * U * roundings * rstd * parts
    if dstream is not None:
        ds = ds + dstream
        tol = tol + U * np.abs(ds)
    return ((ds, (dy * xh).sum(0), dy.sum(0)),
            (tol, 1.01 * U * gamma_roundings * np.abs(dy * xh).sum(0),
             1.01 * U * beta_roundings * np.abs(dy).sum(0)))
