"""The gated sandwich tail and its gradient in 64 bits (numpy), and the error bounds that the
tests hold the kernels to.

u = 2^-24.  A sum over a row has at most c = chain(n) additions on the way of any term, a sum over
rows at most row_chain(rows) (tests/train_bounds.py counts them).  The root of a sum of squares
taken that way, with its product by 1 / n, its sum with eps and rsqrt's two units, is off by e =
u (c / 2 + 8) relative.  Everything below adds up what each term of a formula carries: two
relative errors add, a sum of terms is off by the sum of their bounds and by its own roundings,
relative to the terms' magnitudes and not to what is left when they cancel.
"""
import numpy as np

from train_bounds import chain, row_chain
from train_reference import U


def inv(v, eps):
    return 1.0 / np.sqrt((v * v).mean(1, keepdims=True) + eps)


def wide(factor, rows, n):
    """A factor (None, [1], [n] or [rows, 1]) over all elements."""
    return np.ones((rows, n)) if factor is None else np.broadcast_to(factor, (rows, n))


def stream(b, res, g1, gate, scale, eps1):
    """(out_stream, its bound without the output's rounding)."""
    rows, n = b.shape
    e = U * (chain(n) / 2 + 8)
    z = b * inv(b, eps1) * g1 * wide(gate, rows, n)
    t = wide(scale, rows, n) * res
    out = z + t
    # z: inv, its product with a gate of a row or of all, gamma with a gate of a channel, their
    # product with b
    return out, np.abs(z) * (e + 4 * U) + U * np.abs(t) + U * np.abs(out)


def normed(s, g2, eps2):
    y = s * inv(s, eps2) * g2
    return y, np.abs(y) * (U * (chain(s.shape[1]) / 2 + 8) + 3 * U)


def backward(dn, b, s, g1, g2, gate, scale, res, eps1, eps2, dstream):
    """{name: (value, bound)} of every gradient that the factors have."""
    rows, n = b.shape
    c, cr = chain(n), row_chain(rows)
    e = U * (c / 2 + 8)
    channel = gate is not None and gate.shape == (n,)
    g = np.ones((rows, 1)) if gate is None or channel else np.broadcast_to(gate, (rows, 1))
    k = g1 * gate if channel else g1 * np.ones(n)
    i1, i2 = inv(b, eps1), inv(s, eps2)
    w, vh, xh = dn * g2, s * i2, b * i1
    d = np.zeros_like(w) if dstream is None else dstream
    ds = i2 * (w - vh * (w * vh).mean(1, keepdims=True)) + d
    mean_abs = i2 * i2 * np.abs(w * s).mean(1, keepdims=True)        # what m is at most
    parts = i2 * np.abs(w) + np.abs(vh) * mean_abs + np.abs(d)
    tds = i2 * np.abs(w) * (e + 3 * U) + np.abs(vh) * mean_abs * (U * (c + 8) + 3 * e) + 3 * U * parts

    q = (ds * k * xh).sum(1, keepdims=True)
    mq = i1 * (i2 * np.abs(w * k * b).sum(1, keepdims=True)
               + mean_abs * i2 * np.abs(s * k * b).sum(1, keepdims=True)
               + np.abs(d * k * b).sum(1, keepdims=True))
    tq = mq * (U * (2 * c + 24) + 5 * e)
    db = i1 * (g * ds * k - xh * (g * q) / n)
    tdb = i1 * np.abs(g * k) * (tds + np.abs(ds) * (e + 5 * U)) \
        + np.abs(xh) * i1 * np.abs(g) / n * (tq + mq * (2 * e + 6 * U)) + U * np.abs(db)
    al = wide(scale, rows, n)
    out = {"dblock": (db, tdb), "dresidual": (al * ds, np.abs(al) * (tds + U * np.abs(ds)))}

    p = dn * vh
    out["dgamma_pre"] = p.sum(0), (U * cr + e + 3 * U) * np.abs(p).sum(0)
    a = g * ds * xh
    ta = (np.abs(g * xh) * (tds + np.abs(ds) * (e + 3 * U))).sum(0) + U * cr * np.abs(a).sum(0)
    if channel:
        out["dgamma_post"] = gate * a.sum(0), np.abs(gate) * (ta + U * np.abs(a.sum(0)))
        out["dgate"] = g1 * a.sum(0), np.abs(g1) * (ta + U * np.abs(a.sum(0)))
    else:
        out["dgamma_post"] = a.sum(0), ta
    if gate is not None and not channel:
        if gate.shape == (1,):
            out["dgate"] = q.sum().reshape(1), (tq.sum() + U * cr * np.abs(q).sum()).reshape(1)
        else:
            out["dgate"] = q, tq
    if scale is not None and res is not None:
        r = ds * res
        tr = np.abs(res) * (tds + 2 * U * np.abs(ds))
        if scale.shape == (1,) and n > 1:
            out["dres_scale"] = (r.sum().reshape(1),
                                 (tr.sum() + U * (cr + c) * np.abs(r).sum()).reshape(1))
        else:
            out["dres_scale"] = r.sum(0), tr.sum(0) + U * cr * np.abs(r).sum(0)
    return out
