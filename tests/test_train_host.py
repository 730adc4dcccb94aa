"""The training operations without a GPU: refusals of the C entry points and of the
torch helpers, and the 64-bit reference against known answers and differences."""
import ctypes

import numpy as np
import pytest
import torch

import train_reference as ref
from dual_epsilon_sandwich_gb300 import _build, mrn

STEP = 0x100000000
A, B, C, D, E, F, G, H, I, J, K, W = (0x7F0000000000 + i * STEP for i in range(12))


@pytest.fixture(scope="module", autouse=True)
def library():
    _build.build()
    return mrn.lib()


def ln(x=A, g=G, b=H, y=B, m=I, r=J, rows=4, n=64, eps=1e-5, dt=mrn.MRN_F32):
    return mrn.mrn_layernorm(x, g, b, y, m, r, rows, n, eps, dt, 0)


def da(x=A, r=B, o=C, rng=K, site=0, p=0.1, rows=4, n=64, dt=mrn.MRN_F32):
    return mrn.mrn_dropout_add(x, r, o, rng, site, p, rows, n, dt, 0)


def dln(x=A, res=B, g=G, b=H, s=C, o=D, m=I, r=J, rng=K, p=0.1, rows=4, n=64, eps=1e-5,
        dt=mrn.MRN_F32):
    return mrn.mrn_dropout_add_layernorm(x, res, g, b, s, o, m, r, rng, 0, p, rows, n, eps, dt, 0)


def lnb(dy=A, x=B, g=G, m=I, r=J, ds=C, dx=D, dg=H, db=K, w=W, wb=1 << 40, rows=4, n=64,
        dt=mrn.MRN_F32):
    return mrn.mrn_layernorm_backward(dy, x, g, m, r, ds, dx, dg, db, w, wb, rows, n, dt, 0)


def dlnb(dy=A, s=B, g=G, m=I, r=J, ds=C, dx=D, dr=E, dg=H, db=K, rng=F, p=0.1, w=W, wb=1 << 40,
         rows=4, n=64, dt=mrn.MRN_F32):
    return mrn.mrn_dropout_add_layernorm_backward(dy, s, g, m, r, ds, dx, dr, dg, db, rng, 0, p,
                                                  w, wb, rows, n, dt, 0)


def rmb(dy=A, x=B, g=G, ds=C, dx=D, dg=H, w=W, wb=1 << 40, rows=4, n=64, eps=1e-5,
        dt=mrn.MRN_F32):
    return mrn.mrn_rmsnorm_backward(dy, x, g, ds, dx, dg, w, wb, rows, n, eps, dt, 0)


ALL = (ln, da, dln, lnb, dlnb, rmb)


@pytest.mark.parametrize("call", ALL)
def test_sizes_types(call):
    assert call(n=0) == mrn.MRN_ERR_INVALID_SIZE
    assert call(rows=-1) == mrn.MRN_ERR_INVALID_SIZE
    assert call(rows=2 ** 62) == mrn.MRN_ERR_INVALID_SIZE
    assert call(n=2 ** 62) == mrn.MRN_ERR_INVALID_SIZE
    assert call(dt=mrn.MRN_F16) == mrn.MRN_ERR_UNSUPPORTED_DTYPE
    assert call(dt=9) == mrn.MRN_ERR_UNSUPPORTED_DTYPE
    assert mrn.mrn_launch_count() == 0


@pytest.mark.parametrize("call", (ln, dln, rmb))
def test_eps(call):
    for eps in (0.0, -1e-5, float("inf"), float("nan")):
        assert call(eps=eps) == mrn.MRN_ERR_INVALID_EPS


@pytest.mark.parametrize("call", (da, dln, dlnb))
def test_probability(call):
    for p in (-0.1, 1.0001, float("inf"), float("nan")):
        assert call(p=p) == mrn.MRN_ERR_INVALID_EPS
    assert call(rng=None) == mrn.MRN_ERR_NULL_POINTER     # needed from p = 2^-17 on
    assert call(rng=K + 4 if call is not dlnb else F + 4) == mrn.MRN_ERR_MISALIGNED


REQUIRED = {ln: ("x", "g", "y"), da: ("x", "o"), dln: ("x", "res", "g", "s", "o"),
            lnb: ("dy", "x", "g", "m", "r", "dx", "dg", "w"),
            dlnb: ("dy", "s", "g", "m", "r", "dx", "dr", "dg", "w"),
            rmb: ("dy", "x", "g", "dx", "dg", "w")}


@pytest.mark.parametrize("call", ALL)
def test_required_pointers(call):
    for name in REQUIRED[call]:
        assert call(**{name: None}) == mrn.MRN_ERR_NULL_POINTER, name
    if call in (ln, dln):                                  # both statistics or neither
        assert call(m=None) == mrn.MRN_ERR_NULL_POINTER
        assert call(r=None) == mrn.MRN_ERR_NULL_POINTER
    assert mrn.mrn_launch_count() == 0


@pytest.mark.parametrize("call", ALL)
def test_alignment_of_pointers(call):
    import inspect
    skip = {"rows", "n", "eps", "dt", "p", "wb", "site"}
    for name, par in inspect.signature(call).parameters.items():
        if name not in skip:
            assert call(**{name: par.default + 2}) == mrn.MRN_ERR_MISALIGNED, name
            if name == "w":
                assert call(w=W + 8) == mrn.MRN_ERR_MISALIGNED


def test_overlaps():
    part = 16
    # a row output may be a row input, never part of one, nor anything else
    assert ln(y=A + part) == mrn.MRN_ERR_ALIASING
    assert ln(y=G) == mrn.MRN_ERR_ALIASING
    assert ln(y=H + part) == mrn.MRN_ERR_ALIASING
    assert ln(m=J + 4) == mrn.MRN_ERR_ALIASING
    assert ln(m=A) == mrn.MRN_ERR_ALIASING
    assert ln(r=B + 8) == mrn.MRN_ERR_ALIASING
    assert da(o=A + part) == mrn.MRN_ERR_ALIASING
    assert da(o=B - part) == mrn.MRN_ERR_ALIASING
    assert da(rng=C + 8) == mrn.MRN_ERR_ALIASING
    assert dln(s=C, o=C) == mrn.MRN_ERR_ALIASING
    assert dln(s=A, o=A) == mrn.MRN_ERR_ALIASING
    assert dln(o=B + part) == mrn.MRN_ERR_ALIASING
    assert dln(rng=D) == mrn.MRN_ERR_ALIASING
    for call in (lnb, dlnb, rmb):
        assert call(dx=A + part) == mrn.MRN_ERR_ALIASING
        assert call(dx=C + part) == mrn.MRN_ERR_ALIASING
        assert call(dg=A) == mrn.MRN_ERR_ALIASING
        assert call(dg=G) == mrn.MRN_ERR_ALIASING
        assert call(w=B) == mrn.MRN_ERR_ALIASING
        assert call(w=D - 16) == mrn.MRN_ERR_ALIASING
        assert call(dg=W + 16) == mrn.MRN_ERR_ALIASING
    assert lnb(db=H) == mrn.MRN_ERR_ALIASING
    assert lnb(m=D) == mrn.MRN_ERR_ALIASING
    assert dlnb(dr=D) == mrn.MRN_ERR_ALIASING
    assert dlnb(dr=D + part) == mrn.MRN_ERR_ALIASING
    assert mrn.mrn_launch_count() == 0


def test_workspace():
    for rows, n in ((1, 1), (4, 64), (16384, 4096), (65536, 16384), (3, 1 << 20)):
        need = mrn.mrn_norm_backward_workspace(rows, n)
        assert 0 < need <= 1 << 30, (rows, n, need)
        for call in (lnb, dlnb, rmb):
            assert call(rows=rows, n=n, wb=need - 1) in (mrn.MRN_ERR_INVALID_SIZE,
                                                         mrn.MRN_ERR_ALIASING)
    assert mrn.mrn_norm_backward_workspace(0, 64) == 0
    for rows, n in ((-1, 4), (4, 0), (4, 2 ** 61)):
        with pytest.raises(mrn.MrnError):
            mrn.mrn_norm_backward_workspace(rows, n)
    assert mrn.lib().mrn_norm_backward_workspace(4, 4, None) == mrn.MRN_ERR_NULL_POINTER
    for call in (lnb, dlnb, rmb):
        assert call(wb=0) == mrn.MRN_ERR_INVALID_SIZE
        assert call(wb=-1) == mrn.MRN_ERR_INVALID_SIZE
    assert mrn.mrn_launch_count() == 0


def test_no_rows():
    assert ln(x=None, g=None, b=None, y=None, m=None, r=None, rows=0) == mrn.MRN_OK
    assert da(x=None, r=None, o=None, rng=None, rows=0) == mrn.MRN_OK
    assert dln(x=None, res=None, g=None, b=None, s=None, o=None, m=None, r=None, rng=None,
               rows=0) == mrn.MRN_OK
    for call in (lnb, dlnb, rmb):      # the weights' gradients are still due
        assert call(rows=0, dg=None) == mrn.MRN_ERR_NULL_POINTER
        assert call(rows=0, dg=H + 2) == mrn.MRN_ERR_MISALIGNED
    assert mrn.mrn_launch_count() == 0


def test_status_texts_name_the_new_causes():
    assert "probability" in mrn.mrn_status_string(mrn.MRN_ERR_INVALID_EPS)
    assert "workspace" in mrn.mrn_status_string(mrn.MRN_ERR_INVALID_SIZE)


def test_helpers_refuse_host_tensors():
    x = torch.zeros(4, 8)
    g = torch.ones(8)
    s = torch.zeros(4)
    for call in (lambda: mrn.layernorm(x, g, g, 1e-5), lambda: mrn.dropout_add(x, x, 0.1, None),
                 lambda: mrn.dropout_add_layernorm(x, x, g, g, 1e-5, 0.1, None),
                 lambda: mrn.layernorm_backward(x, x, g, s, s),
                 lambda: mrn.dropout_add_layernorm_backward(x, x, g, s, s, 0.1, None),
                 lambda: mrn.rmsnorm_backward(x, x, g, 1e-5),
                 lambda: mrn.norm_backward_workspace(x)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(TypeError):
        mrn.layernorm(x.to(torch.float16), g, g, 1e-5)


# ---------------------------------------------------------------------------
# The reference itself
# ---------------------------------------------------------------------------
def test_philox_known_answers():
    """The published test vectors of Philox4x32-10."""
    def words(ctr, key):
        return [int(w[0]) for w in ref.philox_words(
            key[0] | key[1] << 32, ctr[2] | ctr[3] << 32, [ctr[0] | ctr[1] << 32])]
    ones = 0xFFFFFFFF
    assert words((0, 0, 0, 0), (0, 0)) == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    assert words((ones,) * 4, (ones, ones)) == [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]
    assert words((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0)) == \
        [0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1]


def test_mask_share_and_independence():
    """The share kept is 1 - t / 2^16 within five standard deviations, and masks of
    two sites agree as often as independent ones do."""
    rows, n, p = 500, 801, 0.25
    a = ref.keep_mask(rows, n, p, 7, 11, 0)
    b = ref.keep_mask(rows, n, p, 7, 11, 1)
    size = rows * n
    for share, expect in ((a.mean(), 0.75), ((a == b).mean(), 0.75 ** 2 + 0.25 ** 2)):
        assert abs(share - expect) < 5 * np.sqrt(expect * (1 - expect) / size)
    assert not np.array_equal(a, ref.keep_mask(rows, n, p, 8, 11, 0))
    assert np.array_equal(b, ref.keep_mask(rows, n, p, 7, 12, 0))   # offset + site
    assert ref.keep_mask(3, 5, 0.0, 1, 2, 3).all() and not ref.keep_mask(3, 5, 1.0, 1, 2, 3).any()
    assert ref.threshold(0.1) == 6554 and ref.drop_scale(0.5) == 2.0


@pytest.mark.parametrize("rows,n", [(1, 1), (1, 2), (3, 7), (4, 33)])
def test_gradients_against_differences(rows, n):
    g = np.random.default_rng(rows * 100 + n)
    x, dy, ds = (g.standard_normal((rows, n)) for _ in range(3))
    gamma, beta = 1 + 0.1 * g.standard_normal(n), 0.1 * g.standard_normal(n)
    eps = 1e-2

    def rms(v, w):
        return v / np.sqrt((v * v).mean(1, keepdims=True) + eps) * w

    def difference(f, v):
        out = np.empty_like(v)
        for i in np.ndindex(v.shape):
            h = 1e-5
            up, down = v.copy(), v.copy()
            up[i] += h
            down[i] -= h
            out[i] = (f(up) - f(down)) / (2 * h)
        return out

    (_, mean, rstd), _ = ref.layernorm(x, gamma, beta, eps)
    (dx, dg, db), _ = ref.layernorm_backward(dy, x, gamma, mean, rstd, ds)

    def loss(v, w, b):
        return (ref.layernorm(v, w, b, eps)[0][0] * dy).sum() + (v * ds).sum()
    np.testing.assert_allclose(dx, difference(lambda v: loss(v, gamma, beta), x), atol=1e-7)
    np.testing.assert_allclose(dg, difference(lambda w: loss(x, w, beta), gamma), atol=1e-7)
    np.testing.assert_allclose(db, difference(lambda b: loss(x, gamma, b), beta), atol=1e-7)
    (dx, dg), _ = ref.rmsnorm_backward(dy, x, gamma, eps, ds)
    np.testing.assert_allclose(
        dx, difference(lambda v: (rms(v, gamma) * dy).sum() + (v * ds).sum(), x), atol=1e-7)
    np.testing.assert_allclose(dg, difference(lambda w: (rms(x, w) * dy).sum(), gamma), atol=1e-7)
