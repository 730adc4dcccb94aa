"""The training operations in 64 bits (numpy), and the error bounds that the
tests hold the kernels to.

Bounds.  u = 2^-24 is half a step of f32 relative to the value, half(dtype) the
rounding of an output to its type (2^-8 for bf16, u for f32).  A sum over a row
whose longest chain of additions is c has an error of at most c * u * sum|terms|;
no kernel adds more than n / 32 terms in one chain before a tree of at most 16
levels, so c = 16 + n / 32 (and for the sums over rows 48 + rows / 8: a CTA adds
the rows it handles in order, at least 8 CTAs run when there are 8 rows, and each
warp of the join adds its share before a tree of 5 levels).
"""
import numpy as np

U = 2.0 ** -24
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}
TINY = 1e-37     # subnormal results are exact to far less than this


def chain(n):
    return 16 + n / 32


def row_chain(rows):
    return 48 + rows / 8


# ---------------------------------------------------------------------------
# Dropout
# ---------------------------------------------------------------------------
def philox_words(seed, step, groups):
    """The four 32-bit words of each group (uint64 array), Philox4x32-10."""
    low = np.uint64(0xFFFFFFFF)
    s32 = np.uint64(32)
    g = np.asarray(groups, dtype=np.uint64)
    c = [g & low, g >> s32, np.full_like(g, step & 0xFFFFFFFF), np.full_like(g, step >> 32)]
    k0, k1 = seed & 0xFFFFFFFF, seed >> 32
    for _ in range(10):
        a = c[0] * np.uint64(0xD2511F53)
        b = c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> s32) ^ c[1] ^ np.uint64(k0), b & low,
             (a >> s32) ^ c[3] ^ np.uint64(k1), a & low]
        k0 = (k0 + 0x9E3779B9) & 0xFFFFFFFF
        k1 = (k1 + 0xBB67AE85) & 0xFFFFFFFF
    return c


def threshold(p):
    return int(np.floor(p * 65536.0 + 0.5))


def drop_scale(p):
    t = threshold(p)
    return 65536.0 / (65536 - t) if t < 65536 else 0.0


def keep_mask(rows, n, p, seed, offset, site):
    """Truth values [rows, n]: the elements kept."""
    total = rows * n
    step = (offset + site) & (2 ** 64 - 1)
    words = philox_words(seed & (2 ** 64 - 1), step, np.arange((total + 7) // 8))
    lanes = np.empty((len(words[0]), 8), dtype=np.uint64)
    for i, w in enumerate(words):
        lanes[:, 2 * i] = w & np.uint64(0xFFFF)
        lanes[:, 2 * i + 1] = w >> np.uint64(16)
    return (lanes.reshape(-1)[:total] >= np.uint64(threshold(p))).reshape(rows, n)


def dropout(x, p, keep):
    return np.where(keep, x * drop_scale(p), 0.0)


def dropout_add(x, residual, p, keep):
    """(value, bound without the output's rounding): the scale is rounded to f32, the
    product and the sum are rounded once."""
    d = dropout(x, p, keep)
    out = residual + d
    return out, U * (2 * np.abs(d) + np.abs(out))


# ---------------------------------------------------------------------------
# Norms and their gradients
# ---------------------------------------------------------------------------
def layernorm(x, gamma, beta, eps):
    """(y, mean, rstd) and their bounds.  The mean is off by c u mean|x|; that shifts
    every deviation alike, which changes the variance by its square only."""
    n = x.shape[1]
    mean = x.mean(1, keepdims=True)
    d = x - mean
    var = (d * d).mean(1, keepdims=True)
    rstd = 1.0 / np.sqrt(var + eps)
    h = d * rstd
    b = np.zeros_like(gamma) if beta is None else beta
    y = h * gamma + b
    c = chain(n)
    dm = U * (c + 2) * np.abs(x).mean(1, keepdims=True)
    # deviations are rounded once each (2 u in a square), beside the shift by dm
    rel = U * (c / 2 + 8) + 0.5 * dm * dm / (var + eps)
    tol = np.abs(gamma) * rstd * dm + np.abs(h * gamma) * (rel + 4 * U) + 2 * U * np.abs(y)
    return (y, mean[:, 0], rstd[:, 0]), (tol, dm[:, 0], (rstd * rel)[:, 0])


def layernorm_backward(dy, x, gamma, mean, rstd, dstream=None):
    """(dx, dgamma, dbeta) and their bounds, from the forward's f32 mean and rstd."""
    rows, n = x.shape
    rstd = rstd[:, None]
    xh = (x - mean[:, None]) * rstd
    return _backward(dy, xh, gamma, rstd, dstream, chain(n), row_chain(rows), True)


def rmsnorm_backward(dy, x, gamma, eps, dstream=None):
    rows, n = x.shape
    inv = 1.0 / np.sqrt((x * x).mean(1, keepdims=True) + eps)
    dx, dg, _ = (None, None, None)
    (dx, dg, _), (tdx, tdg, _) = _backward(dy, x * inv, gamma, inv, dstream, chain(n),
                                           row_chain(rows) + chain(n), False)
    return (dx, dg), (tdx, tdg)


def _backward(dy, xh, gamma, rstd, dstream, c, cr, centred):
    w = dy * gamma
    c1 = w.mean(1, keepdims=True) if centred else np.zeros_like(rstd)
    c2 = (w * xh).mean(1, keepdims=True)
    ds = rstd * (w - c1 - xh * c2)
    # w, xh and rstd carry a few roundings each (for RMSNorm rstd carries its sum's), the
    # two means c roundings; every difference is taken once
    parts = np.abs(w) + np.abs(w).mean(1, keepdims=True) * centred \
        + np.abs(xh) * np.abs(w * xh).mean(1, keepdims=True)
    tol = rstd * U * (2 * c + 8) * parts
    if dstream is not None:
        ds = ds + dstream
        tol = tol + U * np.abs(dstream)
    tol = tol + 2 * U * np.abs(ds)
    dgamma, dbeta = (dy * xh).sum(0), dy.sum(0)
    return ((ds, dgamma, dbeta),
            (tol, U * (cr + 8) * np.abs(dy * xh).sum(0), U * cr * np.abs(dy).sum(0)))


def check(got, want, tol, dtype, what):
    """got (as float64) against want: the bound tol, then the rounding to dtype."""
    got = np.asarray(got, dtype=np.float64)
    limit = tol + HALF[dtype] * (np.abs(want) + tol) + TINY
    bad = ~(np.abs(got - want) <= limit)
    bad &= ~(np.isnan(got) & np.isnan(want))
    if bad.any():
        i = tuple(int(v[0]) for v in np.nonzero(bad))
        raise AssertionError(f"{what}: {int(bad.sum())} of {got.size} off; at {i} got {got[i]!r}, "
                             f"expected {want[i]!r} +- {limit[i]!r}")
