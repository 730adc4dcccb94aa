"""The training operations on the GPU against their 64-bit reference: LayerNorm, the
residual add with dropout, and the gradients of LayerNorm and RMSNorm."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import train_reference as ref
from dual_epsilon_sandwich_gb300 import mrn

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
DTYPES = ("f32", "bf16")
SEED, OFFSET, SITE = -0x123456789ABCDEF, 0x7FFFFFFFFFFFFFF0, 21   # the step's low half wraps
GUARD = 64

# rows x n: one and two elements, lanes, warps and CTAs left partly idle, odd widths, widths
# of the benchmark, rows over clusters of CTAs and wider than any register tile
SHAPES = [(1, 1), (3, 2), (5, 7), (2, 31), (9, 32), (65, 33), (3, 127), (1300, 64), (700, 130),
          (33, 255), (64, 768), (7, 1023), (33, 1024), (160, 2049), (5, 4096), (4, 4097),
          (3, 6655), (4, 6656), (2, 8200), (3, 16384), (2, 20001), (1, 40000), (2, 70000),
          (1, 131080), (2, 140001), (1, 270001)]
# more rows than SMs: every number of slots per thread and of rows at a time, several turns of a
# CTA and a last one that is not full, one warp and several warps to a row, clusters
SHAPES += [(9999, 3), (5000, 8), (3001, 15), (2500, 100), (1301, 257), (1000, 769), (1001, 1025),
           (333, 1535), (1250, 1544), (700, 3001), (613, 4095), (620, 4096), (457, 5121),
           (461, 6655), (470, 6656), (320, 8191), (161, 12296), (155, 16391), (159, 33000),
           (153, 65544)]


@pytest.fixture(scope="module", autouse=True)
def library(gpu_lib):
    return gpu_lib


class Buf:
    """A device tensor [shape] `shift` elements past a 16-byte boundary, with guard bands."""

    def __init__(self, shape, dtype, values=None, shift=0):
        count = int(np.prod(shape))
        self.raw = torch.full((count + 2 * GUARD + shift,), float("nan"), dtype=dtype,
                              device="cuda")
        self.lo = GUARD + shift
        self.t = self.raw[self.lo:self.lo + count].view(shape)
        if values is not None:
            self.t.copy_(values)

    def guards_hold(self):
        n = self.t.numel()
        return bool(self.raw[:self.lo].isnan().all()) and bool(self.raw[self.lo + n:].isnan().all())


def make(seed, rows, n, dtype, scale=1.0, mean=0.0):
    g = torch.Generator().manual_seed(seed)
    return (mean + scale * torch.randn(rows, n, generator=g)).to(TYPES[dtype])


def weights(seed, n, dtype):
    g = torch.Generator().manual_seed(seed)
    return ((1 + 0.1 * torch.randn(n, generator=g)).to(TYPES[dtype]),
            (0.1 * torch.randn(n, generator=g)).to(TYPES[dtype]))


def f64(t):
    return t.detach().cpu().double().numpy()


def rng_tensor(seed=SEED, offset=OFFSET):
    return torch.tensor([seed, offset], dtype=torch.int64, device="cuda")


def keep_of(rows, n, p):
    return ref.keep_mask(rows, n, p, SEED, OFFSET, SITE)


def run_layernorm(x, gamma, beta, eps, dtype, shift=0):
    """Through guarded buffers; returns (y, mean, rstd) as float64 after the guards' check."""
    rows, n = x.shape
    bx, by = Buf((rows, n), TYPES[dtype], x, shift), Buf((rows, n), TYPES[dtype], None, shift)
    mean, rstd = Buf((rows,), torch.float32), Buf((rows,), torch.float32)
    mrn.layernorm(bx.t, gamma.cuda(), None if beta is None else beta.cuda(), eps, out=by.t,
                  mean=mean.t, rstd=rstd.t)
    torch.cuda.synchronize()
    assert by.guards_hold() and mean.guards_hold() and rstd.guards_hold()
    return f64(by.t), f64(mean.t), f64(rstd.t)


def check_layernorm(got, x, gamma, beta, eps, dtype, what):
    (y, mean, rstd), (ty, tm, tr) = ref.layernorm(
        f64(x), f64(gamma), None if beta is None else f64(beta), float(np.float32(eps)))
    ref.check(got[1], mean, tm, "f32", what + " mean")
    ref.check(got[2], rstd, tr, "f32", what + " rstd")
    ref.check(got[0], y, ty, dtype, what + " y")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,n", SHAPES)
def test_layernorm(rows, n, dtype):
    x = make(rows + n, rows, n, dtype, 2.0, 0.5)
    gamma, beta = weights(n, n, dtype)
    for shift, b in ((0, beta), (1, None)):
        got = run_layernorm(x, gamma, b, 1e-5, dtype, shift)
        check_layernorm(got, x, gamma, b, 1e-5, dtype, f"shift {shift}")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,n", SHAPES)
@pytest.mark.parametrize("p", (0.0, 0.1))
def test_dropout_add_layernorm(rows, n, dtype, p):
    x, res = make(1, rows, n, dtype, 2.0), make(2, rows, n, dtype)
    gamma, beta = weights(3, n, dtype)
    keep = keep_of(rows, n, p)
    want, tol = ref.dropout_add(f64(x), f64(res), p, keep)
    for shift in (0, 1):
        t = TYPES[dtype]
        bs, by = Buf((rows, n), t, None, shift), Buf((rows, n), t, None, shift)
        mean, rstd = Buf((rows,), torch.float32), Buf((rows,), torch.float32)
        mrn.dropout_add_layernorm(Buf((rows, n), t, x, shift).t, Buf((rows, n), t, res, shift).t,
                                  gamma.cuda(), beta.cuda(), 1e-6, p,
                                  rng_tensor() if p else None, site=SITE, out_stream=bs.t,
                                  normed=by.t, mean=mean.t, rstd=rstd.t)
        torch.cuda.synchronize()
        assert bs.guards_hold() and by.guards_hold()
        ref.check(f64(bs.t), want, tol, dtype, "stream")
        if p:
            assert np.array_equal(f64(bs.t)[~keep], f64(res)[~keep])
        # normed is the norm of the stream as stored
        check_layernorm((f64(by.t), f64(mean.t), f64(rstd.t)), bs.t, gamma, beta, 1e-6, dtype,
                        f"shift {shift}")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,n", [(1, 1), (1, 3), (2, 8), (5, 7), (3, 1024), (63, 2049),
                                    (257, 4096)])
@pytest.mark.parametrize("p", (0.0, 1e-6, 0.3, 1.0))
def test_dropout_add(rows, n, dtype, p):
    x, res = make(4, rows, n, dtype, 2.0), make(5, rows, n, dtype)
    keep = keep_of(rows, n, p)
    t = TYPES[dtype]
    for shifts in ((0, 0, 0), (1, 1, 1), (0, 1, 2)):
        bx, br, bo = (Buf((rows, n), t, v, s) for v, s in zip((x, res, None), shifts))
        mrn.dropout_add(bx.t, br.t, p, rng_tensor(), site=SITE, out=bo.t)
        want, tol = ref.dropout_add(f64(x), f64(res), p, keep)
        ref.check(f64(bo.t), want, tol, dtype, f"shifts {shifts}")
        assert np.array_equal(f64(bo.t)[~keep], f64(res)[~keep]) and bo.guards_hold()
        mrn.dropout_add(bx.t, None, p, rng_tensor(), site=SITE, out=bo.t)
        want = ref.dropout(f64(x), p, keep)
        ref.check(f64(bo.t), want, 2 * ref.U * np.abs(want), dtype, "alone")
        assert bo.guards_hold()


def run_backward(kind, dy, x, gamma, mean, rstd, dstream, dtype, p=0.1, bias=True, shift=0,
                 eps=1e-5):
    rows, n = x.shape
    t = TYPES[dtype]
    bdy, bx = Buf((rows, n), t, dy, shift), Buf((rows, n), t, x, shift)
    bd = None if dstream is None else Buf((rows, n), t, dstream, shift).t
    dx, dr = Buf((rows, n), t, None, shift), Buf((rows, n), t, None, shift)
    dg, db = Buf((n,), torch.float32), Buf((n,), torch.float32)
    # NaN in the workspace: nothing of it may be read before it is written
    need = mrn.mrn_norm_backward_workspace(rows, n)
    ws = torch.full((need // 4,), float("nan"), device="cuda").view(torch.uint8)
    if kind == "rms":
        mrn.rmsnorm_backward(bdy.t, bx.t, gamma.cuda(), eps, dstream=bd, dx=dx.t, dgamma=dg.t,
                             workspace=ws)
    elif kind == "ln":
        mrn.layernorm_backward(bdy.t, bx.t, gamma.cuda(), mean, rstd, dstream=bd, dx=dx.t,
                               dgamma=dg.t, dbeta=db.t if bias else None, bias=bias, workspace=ws)
    else:
        mrn.dropout_add_layernorm_backward(
            bdy.t, bx.t, gamma.cuda(), mean, rstd, p, rng_tensor(), site=SITE, dstream=bd, dx=dx.t,
            dresidual=dr.t, dgamma=dg.t, dbeta=db.t if bias else None, bias=bias, workspace=ws)
    torch.cuda.synchronize()
    for b in (dx, dr, dg, db):
        assert b.guards_hold()
    return dx.t, dr.t, dg.t, db.t


def device_stats(x, eps=1e-5):
    """The statistics that the forward keeps (any f32 values do for the gradient)."""
    xd = x.cuda()
    rows, n = x.shape
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    one = torch.ones(n, dtype=x.dtype, device="cuda")
    mrn.layernorm(xd, one, None, eps, mean=mean, rstd=rstd)
    return mean, rstd


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,n", SHAPES)
@pytest.mark.parametrize("kind", ("ln", "drop", "rms"))
def test_backward(kind, rows, n, dtype):
    x, dy = make(6, rows, n, dtype, 1.5, 0.3), make(7, rows, n, dtype)
    gamma, _ = weights(8, n, dtype)
    mean, rstd = device_stats(x)
    for shift, ds, bias in ((0, None, True), (1, make(9, rows, n, dtype), False)):
        d64 = None if ds is None else f64(ds)
        dx, dr, dg, db = run_backward(kind, dy, x, gamma, mean, rstd, ds, dtype, bias=bias,
                                      shift=shift)
        if kind == "rms":
            (wx, wg), (tx, tg) = ref.rmsnorm_backward(f64(dy), f64(x), f64(gamma),
                                                      float(np.float32(1e-5)), d64)
        else:
            (wx, wg, wb), (tx, tg, tb) = ref.layernorm_backward(
                f64(dy), f64(x), f64(gamma), f64(mean), f64(rstd), d64)
            if bias:
                ref.check(f64(db), wb, tb, "f32", f"dbeta shift {shift}")
        ref.check(f64(dg), wg, tg, "f32", f"dgamma shift {shift}")
        if kind == "drop":
            keep = keep_of(rows, n, 0.1)
            ref.check(f64(dr), wx, tx, dtype, f"dresidual shift {shift}")
            s = ref.drop_scale(0.1)
            ref.check(f64(dx), ref.dropout(wx, 0.1, keep),
                      np.where(keep, s * (tx + 2 * ref.U * np.abs(wx)), 0.0), dtype,
                      f"dx shift {shift}")
        else:
            ref.check(f64(dx), wx, tx, dtype, f"dx shift {shift}")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n", (1, 33, 1024, 4097, 20001))
def test_unusual_rows(n, dtype):
    """A constant row, a zero row, a row far from zero, a tiny and a large row."""
    x = make(10, 6, n, dtype)
    x[0] = 3.0
    x[1] = 0.0
    x[2] = (x[2].float() + 1000.0).to(x.dtype)
    x[3] = (x[3].float() * 1e-15).to(x.dtype)
    x[4] = (x[4].float() * 1e12).to(x.dtype)
    gamma, beta = weights(11, n, dtype)
    got = run_layernorm(x, gamma, beta, 1e-5, dtype)
    check_layernorm(got, x, gamma, beta, 1e-5, dtype, "unusual")
    assert np.array_equal(got[0][1], f64(beta))
    if n == 1:
        assert np.array_equal(got[0], np.repeat(f64(beta)[None], 6, 0))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n", (1, 33, 1024, 4097, 20001))
@pytest.mark.parametrize("kind", ("ln", "rms"))
def test_gradients_of_unusual_rows(kind, n, dtype):
    """The same rows, and incoming gradients of zero."""
    x, dy = make(18, 7, n, dtype), make(19, 7, n, dtype)
    x[0], x[1] = 3.0, 0.0
    x[2] = (x[2].float() + 1000.0).to(x.dtype)
    x[3] = (x[3].float() * 1e-15).to(x.dtype)
    x[4] = (x[4].float() * 1e17).to(x.dtype)
    dy[5] = 0.0
    gamma, _ = weights(20, n, dtype)
    mean, rstd = device_stats(x)
    dx, _, dg, db = run_backward(kind, dy, x, gamma, mean, rstd, None, dtype)
    if kind == "rms":
        (wx, wg), (tx, tg) = ref.rmsnorm_backward(f64(dy), f64(x), f64(gamma),
                                                  float(np.float32(1e-5)))
    else:
        (wx, wg, wb), (tx, tg, tb) = ref.layernorm_backward(f64(dy), f64(x), f64(gamma), f64(mean),
                                                            f64(rstd))
        ref.check(f64(db), wb, tb, "f32", "dbeta")
    ref.check(f64(dx), wx, tx, dtype, "dx")
    ref.check(f64(dg), wg, tg, "f32", "dgamma")
    assert not f64(dx)[5].any()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n", (5, 1024, 4097))
def test_infinities_stay_in_their_rows(n, dtype):
    rows = 7
    x, dy = make(12, rows, n, dtype), make(13, rows, n, dtype)
    clean = x.clone()
    x[2, n // 2] = float("nan")
    x[4, n - 1] = float("inf")
    gamma, beta = weights(14, n, dtype)
    got, base = (run_layernorm(v, gamma, beta, 1e-5, dtype)[0] for v in (x, clean))
    mean, rstd = device_stats(x)
    bad = np.array([2, 4])
    good = np.array([0, 1, 3, 5, 6])
    assert np.isnan(got[bad]).any(1).all() and np.array_equal(got[good], base[good])
    dxs = []
    for v in (x, clean):
        m, r = device_stats(v)
        dxs.append(f64(run_backward("ln", dy, v, gamma, m, r, None, dtype)[0]))
    assert np.array_equal(dxs[0][good], dxs[1][good])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n", (40, 1023, 4096))
def test_dropped_values_do_not_reach_the_result(n, dtype):
    rows, p = 9, 0.4
    keep = torch.from_numpy(keep_of(rows, n, p))
    x, res = make(15, rows, n, dtype), make(16, rows, n, dtype)
    poisoned = x.clone()
    poisoned[~keep] = float("nan")
    poisoned[0][~keep[0]] = float("inf")
    gamma, beta = weights(17, n, dtype)
    outs = []
    for v in (x, poisoned):
        a = mrn.dropout_add(v.cuda(), res.cuda(), p, rng_tensor(), site=SITE)
        b = mrn.dropout_add(v.cuda(), None, p, rng_tensor(), site=SITE)
        s, y = mrn.dropout_add_layernorm(v.cuda(), res.cuda(), gamma.cuda(), beta.cuda(), 1e-5, p,
                                         rng_tensor(), site=SITE)
        outs.append([f64(t) for t in (a, b, s, y)])
    for u, v in zip(*outs):
        assert np.isfinite(v).all() and np.array_equal(u, v)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,n", [(5, 33), (40, 1023), (700, 512), (3, 20001), (1501, 1023),
                                    (2000, 99)])
def test_in_place(rows, n, dtype):
    """Every output that may be one of the row inputs gives the bits it gives elsewhere."""
    t = TYPES[dtype]
    x, dy, ds = (make(s, rows, n, dtype).cuda() for s in (20, 21, 22))
    gamma, beta = (w.cuda() for w in weights(23, n, dtype))
    mean, rstd = device_stats(x)
    rng = rng_tensor()

    want = mrn.layernorm(x, gamma, beta, 1e-5)
    y = x.clone()
    assert torch.equal(mrn.layernorm(y, gamma, beta, 1e-5, out=y), want)
    want = mrn.dropout_add(x, dy, 0.2, rng)
    for k in (0, 1):
        v = [x.clone(), dy.clone()]
        assert torch.equal(mrn.dropout_add(v[0], v[1], 0.2, rng, out=v[k]), want)
    want = mrn.dropout_add_layernorm(x, dy, gamma, beta, 1e-5, 0.2, rng)
    for k in (0, 1):
        v = [x.clone(), dy.clone()]
        got = mrn.dropout_add_layernorm(v[0], v[1], gamma, beta, 1e-5, 0.2, rng, out_stream=v[k],
                                        normed=v[1 - k])
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    want = mrn.layernorm_backward(dy, x, gamma, mean, rstd, dstream=ds)
    rwant = mrn.rmsnorm_backward(dy, x, gamma, 1e-5, dstream=ds)
    dwant = mrn.dropout_add_layernorm_backward(dy, x, gamma, mean, rstd, 0.2, rng, dstream=ds)
    for k in range(3):
        v = [dy.clone(), x.clone(), ds.clone()]
        got = mrn.layernorm_backward(v[0], v[1], gamma, mean, rstd, dstream=v[2], dx=v[k])
        assert all(torch.equal(a, b) for a, b in zip(got, want)), k
        v = [dy.clone(), x.clone(), ds.clone()]
        got = mrn.rmsnorm_backward(v[0], v[1], gamma, 1e-5, dstream=v[2], dx=v[k])
        assert all(torch.equal(a, b) for a, b in zip(got, rwant)), k
        v = [dy.clone(), x.clone(), ds.clone()]
        got = mrn.dropout_add_layernorm_backward(v[0], v[1], gamma, mean, rstd, 0.2, rng,
                                                 dstream=v[2], dx=v[k], dresidual=v[(k + 1) % 3])
        assert all(torch.equal(a, b) for a, b in zip(got, dwant)), k


@pytest.mark.parametrize("dtype", DTYPES)
def test_operands_at_different_offsets(dtype):
    rows, n = 37, 1000
    t = TYPES[dtype]
    x, dy = make(24, rows, n, dtype), make(25, rows, n, dtype)
    gamma, beta = weights(26, n, dtype)
    gb, bb = Buf((n,), t, gamma, 1).t, Buf((n,), t, beta, 3).t
    y = Buf((rows, n), t, None, 2)
    mrn.layernorm(Buf((rows, n), t, x, 1).t, gb, bb, 1e-5, out=y.t)
    (want, _, _), (tol, _, _) = ref.layernorm(f64(x), f64(gamma), f64(beta),
                                              float(np.float32(1e-5)))
    ref.check(f64(y.t), want, tol, dtype, "y")
    assert y.guards_hold()
    mean, rstd = device_stats(x)
    dx = Buf((rows, n), t, None, 3)
    _, dg, db = mrn.layernorm_backward(Buf((rows, n), t, dy, 2).t, Buf((rows, n), t, x, 1).t, gb,
                                       mean, rstd, dx=dx.t)
    (wx, wg, wb), (tx, tg, tb) = ref.layernorm_backward(f64(dy), f64(x), f64(gamma), f64(mean),
                                                        f64(rstd))
    ref.check(f64(dx.t), wx, tx, dtype, "dx")
    ref.check(f64(dg), wg, tg, "f32", "dgamma")
    ref.check(f64(db), wb, tb, "f32", "dbeta")
    assert dx.guards_hold()
    # only the weights off their boundary, rows aligned
    got = mrn.layernorm(x.cuda(), gb, bb, 1e-5)
    ref.check(f64(got), want, tol, dtype, "y, weights shifted")


def test_no_rows():
    n = 300
    x = torch.empty(0, n, device="cuda")
    gamma = torch.ones(n, device="cuda")
    stat = torch.empty(0, device="cuda")
    assert mrn.layernorm(x, gamma, None, 1e-5, mean=stat, rstd=stat).shape == x.shape
    assert mrn.dropout_add(x, x, 0.1, rng_tensor()).shape == x.shape
    nan = torch.full((n,), float("nan"), device="cuda")
    _, dg, db = mrn.layernorm_backward(x, x, gamma, stat, stat, dgamma=nan.clone(),
                                       dbeta=nan.clone())
    _, _, dg2, db2 = mrn.dropout_add_layernorm_backward(x, x, gamma, stat, stat, 0.1, rng_tensor(),
                                                        dgamma=nan.clone(), dbeta=nan.clone())
    _, dg3 = mrn.rmsnorm_backward(x, x, gamma, 1e-5, dgamma=nan.clone())
    for v in (dg, db, dg2, db2, dg3):
        assert torch.equal(v, torch.zeros(n, device="cuda"))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,n", [(700, 513), (2000, 128), (400, 4096)])
def test_same_call_same_bits(rows, n, dtype):
    """Twice in a row, on another stream and without programmatic launches."""
    x, dy = make(30, rows, n, dtype).cuda(), make(31, rows, n, dtype).cuda()
    gamma, beta = (w.cuda() for w in weights(32, n, dtype))
    rng = rng_tensor()

    def step():
        mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
        s, y = mrn.dropout_add_layernorm(x, dy, gamma, beta, 1e-5, 0.1, rng, mean=mean, rstd=rstd)
        return (s, y, mean, rstd) + mrn.dropout_add_layernorm_backward(
            dy, s, gamma, mean, rstd, 0.1, rng, dstream=x) + mrn.rmsnorm_backward(dy, x, gamma, 1e-5)

    first = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        second = step()
    side.synchronize()
    assert mrn.mrn_set_launch_options(0) == 0
    try:
        third = step()
    finally:
        mrn.mrn_set_launch_options(mrn.MRN_LAUNCH_PDL)
    torch.cuda.synchronize()
    for a, b, c in zip(first, second, third):
        assert torch.equal(a, b) and torch.equal(a, c)


def test_two_streams_at_once():
    """Calls that overlap in time, each with its own workspace."""
    rows, n = 3000, 1000
    streams = [torch.cuda.Stream() for _ in range(2)]
    x = [make(40 + i, rows, n, "bf16").cuda() for i in range(2)]
    dy = [make(50 + i, rows, n, "bf16").cuda() for i in range(2)]
    gamma = torch.ones(n, dtype=torch.bfloat16, device="cuda")
    want = [mrn.rmsnorm_backward(dy[i], x[i], gamma, 1e-5) for i in range(2)]
    torch.cuda.synchronize()
    ws = [mrn.norm_backward_workspace(x[i]) for i in range(2)]
    out = [(torch.empty_like(x[0]), torch.empty(n, device="cuda")) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                mrn.rmsnorm_backward(dy[i], x[i], gamma, 1e-5, dx=out[i][0], dgamma=out[i][1],
                                     workspace=ws[i])
    torch.cuda.synchronize()
    for i in range(2):
        assert torch.equal(out[i][0], want[i][0]) and torch.equal(out[i][1], want[i][1])


def test_captured_step_draws_new_masks():
    """A captured training step replayed with the generator's offset advanced on the
    device gives what the eager calls with that offset give."""
    rows, n, p = 200, 1023, 0.25
    x, res, dy = (make(s, rows, n, "bf16").cuda() for s in (60, 61, 62))
    gamma, beta = (w.cuda() for w in weights(63, n, "bf16"))
    rng = rng_tensor(5, 100)
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    ws = mrn.norm_backward_workspace(x)

    def step(r):
        s, y = mrn.dropout_add_layernorm(x, res, gamma, beta, 1e-5, p, r, site=2, mean=mean,
                                         rstd=rstd)
        return (s, y) + mrn.dropout_add_layernorm_backward(dy, s, gamma, mean, rstd, p, r, site=2,
                                                           workspace=ws)

    step(rng)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(rng)
        rng[1].add_(7)
    seen = []
    for i in range(3):
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        want = step(rng_tensor(5, 100 + 7 * i))
        assert all(torch.equal(a, b) for a, b in zip(got, want)), i
        seen.append(got[0])
    assert not torch.equal(seen[0], seen[1])
    assert int(rng[1]) == 121


def test_offset_and_site_make_the_counter():
    """Equal offset + site give equal masks; seed, offset and site each change them."""
    x = torch.ones(64, 512, device="cuda")

    def mask(seed, offset, site):
        return mrn.dropout_add(x, None, 0.5, rng_tensor(seed, offset), site=site) != 0

    base = mask(1, 10, 2)
    assert torch.equal(base, mask(1, 8, 4)) and torch.equal(base, mask(1, 12, 0))
    for other in (mask(2, 10, 2), mask(1, 11, 2), mask(1, 10, 3), mask(1 + 2 ** 40, 10, 2),
                  mask(1, 10 + 2 ** 40, 2)):
        agree = (base == other).double().mean().item()
        assert 0.45 < agree < 0.55
    # offset + site wraps modulo 2^64
    assert torch.equal(mask(1, -1, 3), mask(1, 0, 2))


def test_helpers_refuse():
    x = torch.zeros(4, 8, device="cuda")
    g = torch.ones(8, device="cuda")
    s = torch.zeros(4, device="cuda")
    rng = rng_tensor()
    bad = [
        lambda: mrn.layernorm(x.t(), g, g, 1e-5),                      # not contiguous
        lambda: mrn.layernorm(x, g[:4], g, 1e-5),                      # wrong shape
        lambda: mrn.layernorm(x, g.bfloat16(), g, 1e-5),               # mixed types
        lambda: mrn.layernorm(x, g, g.cpu(), 1e-5),                    # host tensor
        lambda: mrn.layernorm(x, g, g, 1e-5, mean=s),                  # one statistic
        lambda: mrn.layernorm(x, g, g, 1e-5, mean=s[:2], rstd=s),
        lambda: mrn.layernorm(x, g, g, 0.0),
        lambda: mrn.layernorm(torch.zeros((), device="cuda"), g, g, 1e-5),
        lambda: mrn.dropout_add(x, x, 0.1, None),                      # no generator
        lambda: mrn.dropout_add(x, x, 0.1, rng.int()),
        lambda: mrn.dropout_add(x, x, 0.1, rng.cpu()),
        lambda: mrn.dropout_add(x, x, -0.1, rng),
        lambda: mrn.dropout_add(x, x, float("nan"), rng),
        lambda: mrn.dropout_add(x, x[:2], 0.1, rng),
        lambda: mrn.dropout_add_layernorm(x, x, g, g, 1e-5, 0.1, rng, out_stream=x, normed=x),
        lambda: mrn.layernorm_backward(x, x, g, None, None),
        lambda: mrn.layernorm_backward(x, x, g, s, s.double()),
        lambda: mrn.layernorm_backward(x, x, g, s, s, dgamma=g.bfloat16()),
        lambda: mrn.layernorm_backward(x, x, g, s, s,
                                       workspace=torch.empty(4, dtype=torch.uint8, device="cuda")),
        lambda: mrn.rmsnorm_backward(x, x, g, -1.0),
    ]
    for i, call in enumerate(bad):
        with pytest.raises((ValueError, TypeError, mrn.MrnError)):
            call()
            pytest.fail(f"call {i} was accepted")


def test_a_training_step_against_autograd():
    """A block's two tails forward and back -- dropout, residual add, LayerNorm, twice --
    against autograd in 64 bits over the same masks."""
    rows, n, p, eps = 37, 1000, 0.2, 1e-5
    gen = torch.Generator().manual_seed(70)
    a, b, r0, dlast = (torch.randn(rows, n, generator=gen) for _ in range(4))
    w = [weights(71 + i, n, "f32") for i in range(2)]
    rng = rng_tensor(9, 4)
    cu = [t.cuda() for t in (a, b, r0, dlast)]
    m = [(torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")) for _ in range(2)]
    s1, y1 = mrn.dropout_add_layernorm(cu[0], cu[2], w[0][0].cuda(), w[0][1].cuda(), eps, p, rng,
                                       site=0, mean=m[0][0], rstd=m[0][1])
    block = mrn.dropout_add(y1, cu[1], p, rng, site=1)       # stands for the sub-block
    s2, y2 = mrn.dropout_add_layernorm(block, s1, w[1][0].cuda(), w[1][1].cuda(), eps, p, rng,
                                       site=2, mean=m[1][0], rstd=m[1][1])
    dblock, ds1, dg1, db1 = mrn.dropout_add_layernorm_backward(cu[3], s2, w[1][0].cuda(), *m[1], p,
                                                               rng, site=2)
    dy1 = mrn.dropout_add(dblock, None, p, rng, site=1)
    da, dr0, dg0, db0 = mrn.dropout_add_layernorm_backward(dy1, s1, w[0][0].cuda(), *m[0], p, rng,
                                                           site=0, dstream=ds1)
    leaves = [t.double().requires_grad_() for t in (a, b, r0, w[0][0], w[0][1], w[1][0], w[1][1])]
    A, B, R, G0, B0, G1, B1 = leaves
    masks = [torch.from_numpy(ref.keep_mask(rows, n, p, 9, 4, s)) for s in range(3)]
    k = ref.drop_scale(p)

    def norm(v, g, c):
        d = v - v.mean(1, keepdim=True)
        return d / torch.sqrt((d * d).mean(1, keepdim=True) + eps) * g + c

    S1 = R + A * masks[0] * k
    Y1 = norm(S1, G0, B0)
    BL = B + Y1 * masks[1] * k
    S2 = S1 + BL * masks[2] * k
    Y2 = norm(S2, G1, B1)
    Y2.backward(dlast.double())
    # f32 all the way: a few hundred roundings of values of order one to ten
    for got, want in ((y2, Y2.detach()), (da, A.grad), (dblock * 1.0, None), (dr0, R.grad),
                      (dg0, G0.grad), (db0, B0.grad), (dg1, G1.grad), (db1, B1.grad)):
        if want is not None:
            scale = float(want.abs().max())
            assert float((got.cpu().double() - want).abs().max()) <= 512 * ref.U * scale
    # the sub-block's other summand has the gradient of the block's input
    scale = float(B.grad.abs().max())
    assert float((dblock.cpu().double() - B.grad).abs().max()) <= 512 * ref.U * scale


def test_sandwich_gradient_from_two_calls():
    """norm_residual_norm's gradient: rmsnorm_backward at the stream, then at the block's
    output, against autograd in 64 bits."""
    rows, n = 21, 777
    gen = torch.Generator().manual_seed(80)
    b, r, dn, ds = (torch.randn(rows, n, generator=gen) for _ in range(4))
    gp, gq = weights(81, n, "f32")[0], weights(82, n, "f32")[0]
    stream, _ = mrn.norm_residual_norm(b.cuda(), r.cuda(), gp.cuda(), gq.cuda(), 1e-8, 1e-5)
    dr, dgq = mrn.rmsnorm_backward(dn.cuda(), stream, gq.cuda(), 1e-5, dstream=ds.cuda())
    db, dgp = mrn.rmsnorm_backward(dr, b.cuda(), gp.cuda(), 1e-8)
    leaves = [t.double().requires_grad_() for t in (b, r, gp, gq)]
    B, R, GP, GQ = leaves
    S = B / torch.sqrt((B * B).mean(1, keepdim=True) + 1e-8) * GP + R
    N = S / torch.sqrt((S * S).mean(1, keepdim=True) + 1e-5) * GQ
    ((N * dn.double()).sum() + (S * ds.double()).sum()).backward()
    for got, leaf in ((db, B), (dr, R), (dgp, GP), (dgq, GQ)):
        scale = float(leaf.grad.abs().max())
        assert float((got.cpu().double() - leaf.grad).abs().max()) <= 512 * ref.U * scale


def test_launches_are_counted():
    x = torch.randn(8, 64, device="cuda")
    g = torch.ones(64, device="cuda")
    before = mrn.mrn_launch_count()
    mrn.layernorm(x, g, g, 1e-5)
    mrn.dropout_add(x, x, 0.1, rng_tensor())
    assert mrn.mrn_launch_count() == before + 2


def test_elements_past_32_bits():
    """More than 2^31 elements: the last rows give what they give alone, and their masks are
    those of their element numbers."""
    rows, n, p = 70001, 32771, 0.25
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GB of device memory")
    x = torch.empty(rows, n, dtype=torch.bfloat16, device="cuda")
    x.normal_(generator=torch.Generator(device="cuda").manual_seed(90))
    gamma, beta = (w.cuda() for w in weights(91, n, "bf16"))
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    out = mrn.layernorm(x, gamma, beta, 1e-5, mean=mean, rstd=rstd)
    alone = f64(mrn.layernorm(x[-200:].clone(), gamma, beta, 1e-5))
    # (another grid may take the sums in another order)
    (_, _, _), (tol, _, _) = ref.layernorm(f64(x[-200:]), f64(gamma), f64(beta), 1e-5)
    ref.check(f64(out[-200:]), alone, 2 * tol + ref.HALF["bf16"] * np.abs(alone), "bf16", "last rows")
    mrn.dropout_add(x, None, p, rng_tensor(), site=SITE, out=out)
    first = (rows - 2) * n // 8
    words = ref.philox_words(SEED & (2 ** 64 - 1), (OFFSET + SITE) & (2 ** 64 - 1),
                             np.arange(first, (rows * n + 7) // 8))
    lanes = np.stack([v for w in words for v in (w & np.uint64(0xFFFF), w >> np.uint64(16))], 1)
    keep = (lanes.reshape(-1) >= ref.threshold(p))[(rows - 2) * n - first * 8:][:2 * n]
    got = f64(out[-2:]).reshape(-1)
    assert not got[~keep].any()
    want = f64(x[-2:]).reshape(-1) * ref.drop_scale(p)
    ref.check(got[keep], want[keep], 2 * ref.U * np.abs(want[keep]), "bf16", "last rows kept")
    # the gradient's last rows: dx from their own statistics
    dx, _, _ = mrn.layernorm_backward(x, x, gamma, mean, rstd, dx=out)
    (want, _, _), (tol, _, _) = ref.layernorm_backward(
        f64(x[-3:]), f64(x[-3:]), f64(gamma), f64(mean[-3:]), f64(rstd[-3:]))
    ref.check(f64(dx[-3:]), want, tol, "bf16", "dx of the last rows")


def test_graphs_that_share_a_workspace():
    """Two captured gradients with one workspace, replayed one after the other on one stream."""
    shapes = [(300, 1000), (2000, 257)]
    x = [make(92 + i, r, n, "f32").cuda() for i, (r, n) in enumerate(shapes)]
    dy = [make(94 + i, r, n, "f32").cuda() for i, (r, n) in enumerate(shapes)]
    gamma = [weights(96 + i, n, "f32")[0].cuda() for i, (_, n) in enumerate(shapes)]
    ws = max((mrn.norm_backward_workspace(t) for t in x), key=lambda t: t.numel())
    want = [mrn.rmsnorm_backward(dy[i], x[i], gamma[i], 1e-5, workspace=ws) for i in range(2)]
    want = [[t.clone() for t in w] for w in want]
    graphs, outs = [], []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(mrn.rmsnorm_backward(dy[i], x[i], gamma[i], 1e-5, workspace=ws))
        graphs.append(g)
    ws.fill_(255)                        # NaN: nothing of an earlier call may be read
    for i in (0, 1, 1, 0, 0, 1):
        for t in outs[i]:
            t.fill_(float("nan"))
        graphs[i].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs[i], want[i])), i


def test_a_large_enough_workspace_serves_smaller_calls():
    x = make(98, 2000, 1000, "bf16").cuda()
    ws = mrn.norm_backward_workspace(x)
    small = x[:50].contiguous()
    gamma = torch.ones(1000, dtype=torch.bfloat16, device="cuda")
    a = mrn.rmsnorm_backward(small, small, gamma, 1e-5, workspace=ws)
    b = mrn.rmsnorm_backward(small, small, gamma, 1e-5)
    assert all(torch.equal(u, v) for u, v in zip(a, b))
    with pytest.raises(mrn.MrnError):
        mrn.rmsnorm_backward(x, x, gamma, 1e-5, workspace=mrn.norm_backward_workspace(small))


def test_unsigned_generator_state():
    x = torch.ones(16, 64, device="cuda")
    signed = rng_tensor(-5, -9)
    assert torch.equal(mrn.dropout_add(x, None, 0.5, signed),
                       mrn.dropout_add(x, None, 0.5, signed.view(torch.uint64)))


def test_threads_calling_at_once():
    """First calls of a shape from several threads, each on its own stream."""
    import threading
    rows, n = 500, 1411
    x = [make(100 + i, rows, n, "bf16").cuda() for i in range(4)]
    gamma, beta = (w.cuda() for w in weights(104, n, "bf16"))
    torch.cuda.synchronize()
    got = [None] * 4

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
            y = mrn.layernorm(x[i], gamma, beta, 1e-5, mean=mean, rstd=rstd)
            got[i] = (y, *mrn.layernorm_backward(x[i], x[i], gamma, mean, rstd))
            torch.cuda.current_stream().synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for i in range(4):
        mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
        y = mrn.layernorm(x[i], gamma, beta, 1e-5, mean=mean, rstd=rstd)
        want = (y, *mrn.layernorm_backward(x[i], x[i], gamma, mean, rstd))
        assert all(torch.equal(a, b) for a, b in zip(got[i], want)), i


def test_a_cluster_whose_messages_are_late_stops_and_recovers():
    """The launch option that makes the first wait of a cluster expect bytes that never come:
    the calls return, the kernels stop after about a second, mrn_wait_timeouts() reports them,
    and the next calls are exact."""
    import time
    rows, n = 3, 16384
    x, dy = make(110, rows, n, "f32"), make(111, rows, n, "f32")
    gamma, beta = weights(112, n, "f32")
    mean, rstd = device_stats(x)
    xd, dyd, gd, bd = x.cuda(), dy.cuda(), gamma.cuda(), beta.cuda()
    assert mrn.mrn_wait_timeouts() == 0
    torch.cuda.synchronize()
    assert mrn.mrn_set_launch_options(mrn.MRN_LAUNCH_PDL | mrn.MRN_LAUNCH_TEST_WAIT_TIMEOUT) == 0
    try:
        t0 = time.perf_counter()
        mrn.layernorm(xd, gd, bd, 1e-5)
        mrn.layernorm_backward(dyd, xd, gd, mean, rstd)
        torch.cuda.synchronize()
        seconds = time.perf_counter() - t0
    finally:
        mrn.mrn_set_launch_options(mrn.MRN_LAUNCH_PDL)
    assert mrn.mrn_wait_timeouts() >= 2 and seconds < 30, seconds
    got = run_layernorm(x, gamma, beta, 1e-5, "f32")
    check_layernorm(got, x, gamma, beta, 1e-5, "f32", "after a timeout")
    dx, _, dg, _ = run_backward("ln", dy, x, gamma, mean, rstd, None, "f32")
    (wx, wg, _), (tx, tg, _) = ref.layernorm_backward(f64(dy), f64(x), f64(gamma), f64(mean),
                                                      f64(rstd))
    ref.check(f64(dx), wx, tx, "f32", "dx after a timeout")
    ref.check(f64(dg), wg, tg, "f32", "dgamma after a timeout")
    assert mrn.mrn_wait_timeouts() == 0


FIRST_CALLS_CAPTURED = """
import torch
from dual_epsilon_sandwich_gb300 import mrn
x = torch.randn(40, 20001, device="cuda")
dy, res = torch.randn_like(x), torch.randn_like(x)
g, b = torch.rand(20001, device="cuda"), torch.rand(20001, device="cuda")
mean, rstd = torch.empty(40, device="cuda"), torch.empty(40, device="cuda")
rng = torch.tensor([3, 4], device="cuda")
stream, normed, dx, dres = (torch.empty_like(x) for _ in range(4))
dg, db = torch.empty_like(g), torch.empty_like(g)
ws = mrn.norm_backward_workspace(x)

def step():
    mrn.dropout_add_layernorm(x, res, g, b, 1e-5, 0.1, rng, out_stream=stream, normed=normed,
                              mean=mean, rstd=rstd)
    mrn.dropout_add_layernorm_backward(dy, stream, g, mean, rstd, 0.1, rng, dx=dx, dresidual=dres,
                                       dgamma=dg, dbeta=db, workspace=ws)
    return [t.clone() for t in (stream, normed, dx, dres, dg, db)]

torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = step()
graph.replay()
torch.cuda.synchronize()
assert all(torch.equal(u, v) for u, v in zip(got, step()))
print("same")
"""


def test_first_calls_of_a_process_captured():
    """What the library asks of a kernel at its first call may be asked inside a capture."""
    out = subprocess.run([sys.executable, "-c", FIRST_CALLS_CAPTURED], cwd=ROOT, timeout=300,
                         capture_output=True, text=True)
    assert out.returncode == 0 and out.stdout.strip() == "same", out.stderr[-2000:]
