"""Paths of the training operations that the shapes of tests/test_gpu_train.py leave to one
combination of offset, stream gradient and bias, held to tight bounds; single large elements
at the places where a row is cut; and more than 2^31 elements through the fused operations."""
import numpy as np
import pytest
import torch

import train_bounds as tight
import train_reference as ref
from dual_epsilon_sandwich_gb300 import mrn
from test_gpu_train import (DTYPES, OFFSET, SEED, SITE, TYPES, device_stats, f64, keep_of, make,
                            rng_tensor, run_backward, run_layernorm, weights)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def library(gpu_lib):
    return gpu_lib


# rows that share a warp (1 to 4 slots a thread, up to 128 rows to a CTA), few rows, one CTA (2
# to 4 slots), clusters, rows wider than a tile; aligned pitches and odd ones
SHAPES = [(128, 8), (100, 5), (2000, 8), (1300, 64), (33, 255), (700, 513), (400, 768), (400, 769),
          (1001, 1024), (5, 2048), (4, 6656), (200, 1544), (400, 4096), (400, 4095), (170, 6656),
          (161, 6655), (160, 8192), (160, 16384), (161, 16391), (3, 33000), (9, 65544),
          (2, 140001)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,n", SHAPES)
@pytest.mark.parametrize("kind,p", (("ln", 0.0), ("drop", 0.1), ("drop", 0.0), ("rms", 0.0)))
def test_offset_stream_gradient_and_bias(kind, p, rows, n, dtype):
    """Aligned and shifted by an element, with and without a stream's gradient and a bias."""
    x, dy = make(6, rows, n, dtype, 1.5, 0.3), make(7, rows, n, dtype)
    gamma, _ = weights(8, n, dtype)
    mean, rstd = device_stats(x)
    keep, scale = keep_of(rows, n, p), ref.drop_scale(p)
    for dstream in (None, make(9, rows, n, dtype)):
        d64 = None if dstream is None else f64(dstream)
        if kind == "rms":
            (wx, wg), (tx, tg) = tight.rmsnorm_backward(f64(dy), f64(x), f64(gamma),
                                                        float(np.float32(1e-5)), d64)
        else:
            (wx, wg, wb), (tx, tg, tb) = tight.layernorm_backward(
                f64(dy), f64(x), f64(gamma), f64(mean), f64(rstd), d64)
        for shift, bias in ((0, True), (0, False), (1, True), (1, False)):
            if kind == "rms" and not bias:
                continue
            dx, dr, dg, db = run_backward(kind, dy, x, gamma, mean, rstd, dstream, dtype, p=p,
                                          bias=bias, shift=shift)
            what = f"stream {dstream is not None} shift {shift} bias {bias}"
            ref.check(f64(dg), wg, tg, "f32", "dgamma " + what)
            if kind != "rms" and bias:
                ref.check(f64(db), wb, tb, "f32", "dbeta " + what)
            else:
                assert np.isnan(f64(db)).all()               # (not written)
            if kind != "drop":
                ref.check(f64(dx), wx, tx, dtype, "dx " + what)
                continue
            ref.check(f64(dr), wx, tx, dtype, "dresidual " + what)
            ref.check(f64(dx), ref.dropout(wx, p, keep),
                      np.where(keep, scale * (tx + 2 * ref.U * np.abs(wx)), 0.0), dtype,
                      "dx " + what)
            assert not f64(dx)[~keep].any()


def cuts(n):
    """Columns at a row's ends and on both sides of where slots, warps and CTAs begin."""
    c = {0, 1, 6, 7, 8, 9, n // 2, n - 9, n - 8, n - 7, n - 2, n - 1}
    for step in (256, 512, 768, 1024, 2048, 4096, 8192, 16384, 32768, 65536):
        for k in (1, 2, 3):
            c |= {k * step - 1, k * step, k * step + 1, k * step + 7, k * step + 8}
    return sorted(j for j in c if 0 <= j < n)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shift", (0, 1))
@pytest.mark.parametrize("n", (1000, 4095, 8192, 16384, 16391, 33000, 65537, 131071, 131080, 140001))
def test_every_element_of_a_row_counts_once(n, shift, dtype):
    """One row per cut: a large value there and zeros elsewhere, where an element lost or taken
    twice is a share of the sums that no bound lets pass; sums and products are exact."""
    cols = torch.tensor(cuts(n))
    rows = len(cols)
    at = torch.arange(rows), cols
    big = 2.0 ** 12
    x = torch.zeros(rows, n)
    x[at] = big
    x = x.to(TYPES[dtype])
    one = torch.ones(n, dtype=TYPES[dtype])
    zero = torch.zeros(n, dtype=TYPES[dtype])
    y, mean, rstd = run_layernorm(x, one, zero, 1e-5, dtype, shift)
    assert np.array_equal(mean, np.full(rows, float(np.float32(big) / np.float32(n))))
    (wy, _, wr), _ = ref.layernorm(f64(x), f64(one), f64(zero), 1e-5)
    np.testing.assert_allclose(rstd, wr, rtol=1e-5)
    np.testing.assert_allclose(y[at], wy[at], rtol=2 * ref.HALF[dtype] + 1e-5)

    # a gradient that is one at the cut: its sums are w = 1 and w xh = xh there
    dy = torch.zeros(rows, n)
    dy[at] = 1.0
    dy = dy.to(TYPES[dtype])
    stat = torch.zeros(rows, device="cuda"), torch.full((rows,), 0.5, device="cuda")
    dx, _, dg, db = run_backward("ln", dy, x, one, *stat, None, dtype, shift=shift)
    xh = big * 0.5
    want = np.full((rows, n), -0.5 / n)
    want[at] = 0.5 * (1 - 1 / n - xh * xh / n)
    np.testing.assert_allclose(f64(dx), want, rtol=2 * ref.HALF[dtype] + 1e-5)
    count = np.zeros(n)
    count[cols.numpy()] = 1.0
    assert np.array_equal(f64(db), count) and np.array_equal(f64(dg), xh * count)
    dx, _, dg, _ = run_backward("rms", dy, x, one, None, None, None, dtype, shift=shift)
    inv = 1 / np.sqrt(big * big / n + float(np.float32(1e-5)))
    got = f64(dx)
    # (the cut's own gradient is what eps leaves of 1 - x^2 inv^2 / n: nothing but roundings)
    assert (np.abs(got[at]) <= 64 * ref.U * inv * (1 + ref.HALF[dtype])).all()
    got[at] = 0.0
    assert not got.any()
    np.testing.assert_allclose(f64(dg), big * inv * count, rtol=1e-5)


def test_fused_operations_past_32_bits():
    """More than 2^31 elements through the tail and its gradient, and RMSNorm's gradient: the
    last rows against the reference, with the masks of their own element numbers."""
    rows, n, p, last = 70001, 32771, 0.25, 3
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB of device memory")
    gen = torch.Generator(device="cuda").manual_seed(90)
    x, res = (torch.empty(rows, n, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
              for _ in range(2))
    gamma, beta = (w.cuda() for w in weights(91, n, "bf16"))
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    stream, normed = mrn.dropout_add_layernorm(x, res, gamma, beta, 1e-5, p, rng_tensor(),
                                               site=SITE, mean=mean, rstd=rstd)
    first = (rows - last) * n // 8
    words = ref.philox_words(SEED & (2 ** 64 - 1), (OFFSET + SITE) & (2 ** 64 - 1),
                             np.arange(first, (rows * n + 7) // 8))
    lanes = np.stack([v for w in words for v in (w & np.uint64(0xFFFF), w >> np.uint64(16))], 1)
    keep = (lanes.reshape(-1) >= ref.threshold(p))[(rows - last) * n - first * 8:][:last * n]
    keep = keep.reshape(last, n)
    want, tol = ref.dropout_add(f64(x[-last:]), f64(res[-last:]), p, keep)
    ref.check(f64(stream[-last:]), want, tol, "bf16", "stream")
    assert np.array_equal(f64(stream[-last:])[~keep], f64(res[-last:])[~keep])
    (wy, wm, wr), (ty, tm, tr) = tight.layernorm(f64(stream[-last:]), f64(gamma), f64(beta),
                                                 float(np.float32(1e-5)))
    for name, g, w, t, kind in (("normed", normed, wy, ty, "bf16"), ("mean", mean, wm, tm, "f32"),
                                ("rstd", rstd, wr, tr, "f32")):
        ref.check(f64(g[-last:]), w, t, kind, name)

    # the gradients, x in the place of normed's
    dx, dres, _, _ = mrn.dropout_add_layernorm_backward(
        x, stream, gamma, mean, rstd, p, rng_tensor(), site=SITE, dstream=res, dx=normed)
    (wx, _, _), (tx, _, _) = tight.layernorm_backward(
        f64(x[-last:]), f64(stream[-last:]), f64(gamma), f64(mean[-last:]), f64(rstd[-last:]),
        f64(res[-last:]))
    ref.check(f64(dres[-last:]), wx, tx, "bf16", "dresidual")
    s = ref.drop_scale(p)
    ref.check(f64(dx[-last:]), ref.dropout(wx, p, keep),
              np.where(keep, s * (tx + 2 * ref.U * np.abs(wx)), 0.0), "bf16", "dx")
    assert not f64(dx[-last:])[~keep].any()
    dx, _ = mrn.rmsnorm_backward(x, stream, gamma, 1e-5, dstream=res, dx=normed)
    (wx, _), (tx, _) = tight.rmsnorm_backward(f64(x[-last:]), f64(stream[-last:]), f64(gamma),
                                              float(np.float32(1e-5)), f64(res[-last:]))
    ref.check(f64(dx[-last:]), wx, tx, "bf16", "dx of the RMSNorm")
