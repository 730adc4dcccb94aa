"""The gated sandwich tail, its gradient and the operations over many tensors without a GPU:
refusals of the C entry points and of the torch helpers, and the 64-bit reference against
differences."""
import inspect

import numpy as np
import pytest
import torch

import gate_reference as ref
from dual_epsilon_sandwich_gb300 import _build, mrn

STEP = 0x100000000
(B, R, S, Y, DN, DS, DB, DR, G1, G2, GATE, SCALE, DG1, DG2, DGATE, DSCALE, W, NORM) = \
    (0x7F0000000000 + i * STEP for i in range(18))
NONE, SCALAR, CHANNEL, ROW = (mrn.MRN_FACTOR_NONE, mrn.MRN_FACTOR_SCALAR, mrn.MRN_FACTOR_CHANNEL,
                              mrn.MRN_FACTOR_ROW)


@pytest.fixture(scope="module", autouse=True)
def library():
    _build.build()
    return mrn.lib()


def fwd(b=B, res=R, g1=G1, g2=G2, gate=GATE, gk=CHANNEL, sc=SCALE, sk=CHANNEL, s=S, y=Y, rows=4,
        n=64, e1=1e-8, e2=1e-5, dt=mrn.MRN_F32):
    return mrn.mrn_norm_gate_residual_norm(b, res, g1, g2, gate, gk, sc, sk, s, y, rows, n, e1, e2,
                                           dt, 0)


def bwd(dn=DN, ds=DS, b=B, s=S, res=R, g1=G1, g2=G2, gate=GATE, gk=CHANNEL, sc=SCALE, sk=CHANNEL,
        db=DB, dr=DR, dg1=DG1, dg2=DG2, dgate=DGATE, dsc=DSCALE, w=W, wb=1 << 40, rows=4, n=64,
        e1=1e-8, e2=1e-5, dt=mrn.MRN_F32):
    return mrn.mrn_norm_gate_residual_norm_backward(dn, ds, b, s, res, g1, g2, gate, gk, sc, sk, db,
                                                    dr, dg1, dg2, dgate, dsc, w, wb, rows, n, e1,
                                                    e2, dt, 0)


SCALARS = {"rows", "n", "e1", "e2", "dt", "wb", "gk", "sk"}


@pytest.mark.parametrize("call", (fwd, bwd))
def test_sizes_types_eps_and_kinds(call):
    for bad in ({"n": 0}, {"rows": -1}, {"rows": 2 ** 62}, {"n": 2 ** 62}, {"gk": 4}, {"gk": -1},
                {"sk": ROW}, {"sk": 4}, {"sk": -1}):
        assert call(**bad) == mrn.MRN_ERR_INVALID_SIZE, bad
    for dt in (mrn.MRN_F16, 9):
        assert call(dt=dt) == mrn.MRN_ERR_UNSUPPORTED_DTYPE
    for eps in (0.0, -1e-5, float("inf"), float("nan")):
        assert call(e1=eps) == mrn.MRN_ERR_INVALID_EPS
        assert call(e2=eps) == mrn.MRN_ERR_INVALID_EPS
    assert mrn.mrn_launch_count() == 0


def test_row_gradients_past_64_bits():
    """bf16 rows of one element take two bytes each, a gate's gradient four."""
    for rows in (2 ** 62 - 1, 2 ** 61):
        assert bwd(rows=rows, n=1, gk=ROW, dt=mrn.MRN_BF16) == mrn.MRN_ERR_INVALID_SIZE


@pytest.mark.parametrize("call,required", (
    (fwd, ("b", "res", "g1", "g2", "gate", "sc", "s", "y")),
    (bwd, ("dn", "b", "s", "res", "g1", "g2", "gate", "sc", "db", "dr", "dg1", "dg2", "w"))))
def test_required_pointers(call, required):
    for name in required:
        assert call(**{name: None}) == mrn.MRN_ERR_NULL_POINTER, name
    for kind in (SCALAR, ROW):
        assert call(gk=kind, gate=None) == mrn.MRN_ERR_NULL_POINTER
    if call is bwd:     # a gradient of a factor that is not there
        assert call(gk=NONE, gate=None) == mrn.MRN_ERR_NULL_POINTER
        assert call(sk=NONE, sc=None) == mrn.MRN_ERR_NULL_POINTER
    assert mrn.mrn_launch_count() == 0


@pytest.mark.parametrize("call", (fwd, bwd))
def test_alignment_of_pointers(call):
    for name, par in inspect.signature(call).parameters.items():
        if name not in SCALARS:
            assert call(**{name: par.default + 2}) == mrn.MRN_ERR_MISALIGNED, name
    if call is bwd:
        assert call(w=W + 8) == mrn.MRN_ERR_MISALIGNED


def test_overlaps():
    part = 16
    assert fwd(s=B + part) == mrn.MRN_ERR_ALIASING
    assert fwd(y=R - part) == mrn.MRN_ERR_ALIASING
    assert fwd(s=S, y=S) == mrn.MRN_ERR_ALIASING
    assert fwd(s=B, y=B) == mrn.MRN_ERR_ALIASING
    assert fwd(gk=ROW, gate=S + 4 * 64) == mrn.MRN_ERR_ALIASING
    for name in ("g1", "g2", "gate", "sc"):
        assert fwd(**{name: Y + 8}) == mrn.MRN_ERR_ALIASING, name
    assert bwd(db=DR, dr=DR) == mrn.MRN_ERR_ALIASING
    for name in ("dn", "ds", "b", "s", "res"):
        at = inspect.signature(bwd).parameters[name].default
        assert bwd(db=at + part) == mrn.MRN_ERR_ALIASING, name
        assert bwd(dr=at - part) == mrn.MRN_ERR_ALIASING, name
        for out in ("dg1", "dg2", "dgate", "dsc", "w"):
            assert bwd(**{out: at}) == mrn.MRN_ERR_ALIASING, (name, out)
    for name in ("dg1", "dg2", "dgate", "dsc"):
        assert bwd(**{name: W + 16}) == mrn.MRN_ERR_ALIASING
        assert bwd(**{name: G1}) == mrn.MRN_ERR_ALIASING
    assert bwd(dg1=DG2) == mrn.MRN_ERR_ALIASING
    assert mrn.mrn_launch_count() == 0


def test_workspace():
    for rows, n in ((1, 1), (4, 64), (16384, 4096), (65536, 16384), (3, 1 << 20)):
        need = mrn.mrn_norm_gate_backward_workspace(rows, n)
        assert 0 < need <= 3 << 29, (rows, n, need)
    need = mrn.mrn_norm_gate_backward_workspace(4, 64)
    for wb in (need - 1, 0, -1):
        assert bwd(wb=wb) == mrn.MRN_ERR_INVALID_SIZE
    assert mrn.mrn_norm_gate_backward_workspace(0, 64) == 0
    for rows, n in ((-1, 4), (4, 0), (4, 2 ** 61)):
        with pytest.raises(mrn.MrnError):
            mrn.mrn_norm_gate_backward_workspace(rows, n)
    assert mrn.lib().mrn_norm_gate_backward_workspace(4, 4, None) == mrn.MRN_ERR_NULL_POINTER


def test_no_rows():
    none = dict.fromkeys(("b", "res", "g1", "g2", "gate", "sc", "s", "y"))
    assert fwd(rows=0, **none) == mrn.MRN_OK
    for name in ("dg1", "dg2"):      # the weights' gradients are still due
        assert bwd(rows=0, **{name: None}) == mrn.MRN_ERR_NULL_POINTER
        assert bwd(rows=0, **{name: DG1 + 2}) == mrn.MRN_ERR_MISALIGNED
    assert mrn.mrn_launch_count() == 0


# ---------------------------------------------------------------------------
# Lists
# ---------------------------------------------------------------------------
def clip(grads=(B, R), out=(S, Y), counts=(64, 64), dtypes=(0, 0), limit=1.0, norm=NORM, w=W,
         wb=1 << 30):
    return mrn.mrn_clip_grad_norm(grads, out, counts, dtypes, limit, norm, w, wb)


def norm(grads=(B, R), counts=(64, 64), dtypes=(0, 0), norm=NORM, w=W, wb=1 << 30):
    return mrn.mrn_grad_norm(grads, counts, dtypes, norm, w, wb)


@pytest.mark.parametrize("call", (norm, clip))
def test_lists_refused(call):
    for bad, status in (
            ({"norm": None}, mrn.MRN_ERR_NULL_POINTER), ({"w": None}, mrn.MRN_ERR_NULL_POINTER),
            ({"grads": (B, None)}, mrn.MRN_ERR_NULL_POINTER),
            ({"norm": NORM + 2}, mrn.MRN_ERR_MISALIGNED), ({"w": W + 4}, mrn.MRN_ERR_MISALIGNED),
            ({"grads": (B, R + 2)}, mrn.MRN_ERR_MISALIGNED),
            ({"grads": (B, R + 1), "dtypes": (0, 1)}, mrn.MRN_ERR_MISALIGNED),
            ({"counts": (64, -1)}, mrn.MRN_ERR_INVALID_SIZE),
            ({"counts": (2 ** 59, 2 ** 59)}, mrn.MRN_ERR_INVALID_SIZE),
            ({"wb": 7}, mrn.MRN_ERR_INVALID_SIZE), ({"wb": -1}, mrn.MRN_ERR_INVALID_SIZE),
            ({"dtypes": (0, 2)}, mrn.MRN_ERR_UNSUPPORTED_DTYPE),
            ({"dtypes": (7, 0)}, mrn.MRN_ERR_UNSUPPORTED_DTYPE),
            ({"norm": B + 8}, mrn.MRN_ERR_ALIASING), ({"w": R}, mrn.MRN_ERR_ALIASING),
            ({"norm": W + 8}, mrn.MRN_ERR_ALIASING)):
        assert call(**bad) == status, bad
    assert mrn.mrn_launch_count() == 0


def test_clips_refused():
    for limit in (-1.0, float("nan"), -1e-30):
        assert clip(limit=limit) == mrn.MRN_ERR_INVALID_EPS
    four = 4 * 64
    for out in ((S, S), (S, S + four - 4), (S + 4, S), (B + 4, Y), (R, B), (S, B), (R, Y),
                (B, R - 4), (NORM, Y), (S, W + 8), (S, R + four - 4)):
        assert clip(out=out) == mrn.MRN_ERR_ALIASING, out
    assert clip(grads=(B, B), out=(B, B)) == mrn.MRN_ERR_ALIASING      # listed twice, in place
    assert clip(out=(S, None)) == mrn.MRN_ERR_NULL_POINTER
    assert clip(out=(S, Y + 2)) == mrn.MRN_ERR_MISALIGNED
    assert mrn.lib().mrn_clip_grad_norm(None, None, None, None, 2, 1.0, NORM, W, 1 << 30, 0) == \
        mrn.MRN_ERR_NULL_POINTER
    assert mrn.lib().mrn_grad_norm(None, None, None, 1, NORM, W, 1 << 30, 0) == \
        mrn.MRN_ERR_NULL_POINTER
    assert mrn.lib().mrn_grad_norm(None, None, None, -1, NORM, W, 1 << 30, 0) == \
        mrn.MRN_ERR_INVALID_SIZE
    assert mrn.mrn_launch_count() == 0


def test_list_workspace():
    one = mrn.mrn_grad_norm_workspace(1)
    assert 0 < one <= 1 << 16 and mrn.mrn_grad_norm_workspace(0) > 0
    assert one <= mrn.mrn_grad_norm_workspace(5000) <= 6 * one
    for bad in (-1, 2 ** 62):
        with pytest.raises(mrn.MrnError):
            mrn.mrn_grad_norm_workspace(bad)
    assert mrn.lib().mrn_grad_norm_workspace(1, None) == mrn.MRN_ERR_NULL_POINTER


def test_helpers_refuse_host_tensors():
    x, g = torch.zeros(4, 8), torch.ones(8)
    for call in (lambda: mrn.norm_gate_residual_norm(x, x, g, g, g),
                 lambda: mrn.norm_gate_residual_norm_backward(x, x, x, g, g),
                 lambda: mrn.norm_gate_backward_workspace(x), lambda: mrn.grad_norm([x]),
                 lambda: mrn.clip_grad_norm([x, g], 1.0), lambda: mrn.grad_norm_workspace([x])):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    for call in (lambda: mrn.grad_norm([]), lambda: mrn.clip_grad_norm([], 1.0),
                 lambda: mrn.grad_norm_workspace([])):
        with pytest.raises(ValueError, match="empty"):
            call()
    with pytest.raises(TypeError):
        mrn.grad_norm([x.half()])


# ---------------------------------------------------------------------------
# The reference itself
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("rows,n", [(1, 1), (1, 2), (3, 7), (4, 33)])
@pytest.mark.parametrize("kind", ("none", "scalar", "channel", "row"))
def test_gradients_against_differences(rows, n, kind):
    g = np.random.default_rng(rows * 100 + n)
    b, res, dn, ds = (g.standard_normal((rows, n)) for _ in range(4))
    g1, g2 = (1 + 0.1 * g.standard_normal(n) for _ in range(2))
    gate = {"none": None, "scalar": g.standard_normal(1), "channel": g.standard_normal(n),
            "row": g.standard_normal((rows, 1))}[kind]
    scale = {"none": None, "scalar": g.standard_normal(1), "channel": None,
             "row": g.standard_normal(n)}[kind]
    e1, e2 = 1e-2, 2e-2
    v = {"dblock": b, "dresidual": res, "dgamma_post": g1, "dgamma_pre": g2, "dgate": gate,
         "dres_scale": scale}

    def loss(v):
        s, _ = ref.stream(v["dblock"], v["dresidual"], v["dgamma_post"], v["dgate"],
                          v["dres_scale"], e1)
        y, _ = ref.normed(s, v["dgamma_pre"], e2)
        return (y * dn).sum() + (s * ds).sum()

    s, _ = ref.stream(b, res, g1, gate, scale, e1)
    got = ref.backward(dn, b, s, g1, g2, gate, scale, res, e1, e2, ds)
    assert ("dgate" in got) == (gate is not None) and ("dres_scale" in got) == (scale is not None)
    for name, (grad, tol) in got.items():
        assert grad.shape == v[name].shape == tol.shape, name
        for i in np.ndindex(grad.shape):
            up, down = dict(v), dict(v)
            up[name], down[name] = v[name].copy(), v[name].copy()
            up[name][i] += 1e-5
            down[name][i] -= 1e-5
            np.testing.assert_allclose(grad[i], (loss(up) - loss(down)) / 2e-5, atol=2e-7,
                                       err_msg=name)
