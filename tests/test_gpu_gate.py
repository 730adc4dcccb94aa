"""The gated sandwich tail and its gradient on the GPU against their 64-bit reference."""
import os
import subprocess
import sys
import threading
import time

import numpy as np
import pytest
import torch

import gate_reference as gate_ref
import train_reference as ref
from dual_epsilon_sandwich_gb300 import mrn
from test_gpu_train import DTYPES, SHAPES, TYPES, Buf, f64, make, weights

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
E1, E2 = float(np.float32(1e-8)), float(np.float32(1e-5))
GATES = ("none", "scalar", "channel", "row")
SCALES = ("none", "scalar", "channel")
# every pair of factors is met as the shapes go by; the last three shapes have all of them
PAIRS = [(g, s) for g in GATES for s in SCALES]


@pytest.fixture(scope="module", autouse=True)
def library(gpu_lib):
    return gpu_lib


def factors(seed, rows, n, dtype, gate, scale):
    """(gate, res_scale) on the host."""
    g = torch.Generator().manual_seed(seed)
    shape = {"none": None, "scalar": (1,), "channel": (n,), "row": (rows, 1)}
    out = []
    for kind, mean, dev in ((gate, 0.4, 0.3), (scale, 1.0, 0.2)):
        s = shape[kind]
        out.append(None if s is None else (mean + dev * torch.randn(s, generator=g)).to(TYPES[dtype]))
    return out


def maybe(t, f):
    return None if t is None else f(t)


def placed(t, dtype, shift):
    """A copy on the device, `shift` elements past a 16-byte boundary, with guard bands."""
    return maybe(t, lambda v: Buf(tuple(v.shape), TYPES[dtype], v, shift).t)


def run_forward(b, res, g1, g2, gate, scale, dtype, shift=0):
    rows, n = b.shape
    s, y = Buf((rows, n), TYPES[dtype], None, shift), Buf((rows, n), TYPES[dtype], None, shift)
    mrn.norm_gate_residual_norm(placed(b, dtype, shift), placed(res, dtype, shift), g1.cuda(),
                                g2.cuda(), gate=placed(gate, dtype, shift),
                                res_scale=placed(scale, dtype, 0), eps_post=1e-8, eps_pre=1e-5,
                                out_stream=s.t, normed=y.t)
    torch.cuda.synchronize()
    assert s.guards_hold() and y.guards_hold()
    return s.t, y.t


def check_forward(got, b, res, g1, g2, gate, scale, dtype, what):
    s, y = got
    want, tol = gate_ref.stream(f64(b), f64(res), f64(g1), maybe(gate, f64), maybe(scale, f64), E1)
    ref.check(f64(s), want, tol, dtype, what + " stream")
    # normed is the norm of the stream as stored
    want, tol = gate_ref.normed(f64(s), f64(g2), E2)
    ref.check(f64(y), want, tol, dtype, what + " normed")


OUTPUTS = ("dblock", "dresidual", "dgamma_post", "dgamma_pre", "dgate", "dres_scale")


def run_backward(dn, b, s, g1, g2, gate, scale, res, dstream, dtype, shift=0):
    """{name: tensor} through guarded buffers and a workspace of NaN."""
    rows, n = b.shape
    out = {k: Buf((rows, n), TYPES[dtype], None, shift) for k in OUTPUTS[:2]}
    out.update({k: Buf((n,), torch.float32) for k in OUTPUTS[2:4]})
    if gate is not None:
        out["dgate"] = Buf(tuple(gate.shape), torch.float32)
    if scale is not None and res is not None:
        out["dres_scale"] = Buf(tuple(scale.shape), torch.float32)
    need = mrn.mrn_norm_gate_backward_workspace(rows, n)
    ws = torch.full((need // 4,), float("nan"), device="cuda").view(torch.uint8)
    mrn.norm_gate_residual_norm_backward(
        placed(dn, dtype, shift), placed(b, dtype, shift), placed(s, dtype, shift), g1.cuda(),
        g2.cuda(), gate=placed(gate, dtype, shift), res_scale=placed(scale, dtype, 0),
        residual=placed(res, dtype, shift), eps_post=1e-8, eps_pre=1e-5,
        dstream=placed(dstream, dtype, shift), workspace=ws, **{k: v.t for k, v in out.items()})
    torch.cuda.synchronize()
    for k, v in out.items():
        assert v.guards_hold(), k
    return {k: v.t for k, v in out.items()}


def check_backward(got, dn, b, s, g1, g2, gate, scale, res, dstream, dtype, what):
    want = gate_ref.backward(f64(dn), f64(b), f64(s), f64(g1), f64(g2), maybe(gate, f64),
                             maybe(scale, f64), maybe(res, f64), E1, E2, maybe(dstream, f64))
    assert set(got) == set(want)
    for k, (value, tol) in want.items():
        ref.check(f64(got[k]), value, tol, dtype if k in OUTPUTS[:2] else "f32", f"{what} {k}")


def operands(seed, rows, n, dtype):
    b, res = make(seed, rows, n, dtype, 2.0), make(seed + 1, rows, n, dtype)
    return b, res, weights(seed + 2, n, dtype)[0], weights(seed + 3, n, dtype)[0]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("i", range(len(SHAPES)))
def test_forward(i, dtype):
    rows, n = SHAPES[i]
    b, res, g1, g2 = operands(100 + i, rows, n, dtype)
    for j, shift in enumerate((0, 0, 1, 1)):
        pair = PAIRS[(4 * i + j + (dtype == "f32")) % len(PAIRS)]
        gate, scale = factors(j, rows, n, dtype, *pair)
        got = run_forward(b, res, g1, g2, gate, scale, dtype, shift)
        check_forward(got, b, res, g1, g2, gate, scale, dtype, f"{pair} shift {shift}")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("i", range(len(SHAPES)))
def test_backward(i, dtype):
    rows, n = SHAPES[i]
    b, res, g1, g2 = operands(200 + i, rows, n, dtype)
    s, dn, ds = (make(300 + i + k, rows, n, dtype, 1.0 + 0.2 * k) for k in range(3))
    for j, (shift, d, r) in enumerate(((0, ds, res), (0, None, None), (1, ds, None), (1, None, res))):
        pair = PAIRS[(5 * i + j + 3 * (dtype == "f32")) % len(PAIRS)]
        gate, scale = factors(j, rows, n, dtype, *pair)
        got = run_backward(dn, b, s, g1, g2, gate, scale, r, d, dtype, shift)
        check_backward(got, dn, b, s, g1, g2, gate, scale, r, d, dtype,
                       f"{pair} shift {shift} stream {d is not None} residual {r is not None}")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,n", [(3, 16), (100, 5), (700, 130), (300, 1000), (4, 6656),
                                    (310, 4096), (320, 4095), (155, 16391), (5, 33000),
                                    (2, 270001), (400, 1024), (350, 2048), (330, 8192), (900, 512),
                                    (320, 1536)])
def test_every_pair_of_factors(rows, n, dtype):
    b, res, g1, g2 = operands(1, rows, n, dtype)
    s, dn, ds = (make(10 + k, rows, n, dtype) for k in range(3))
    for pair in PAIRS:
        gate, scale = factors(7, rows, n, dtype, *pair)
        got = run_forward(b, res, g1, g2, gate, scale, dtype)
        check_forward(got, b, res, g1, g2, gate, scale, dtype, str(pair))
        got = run_backward(dn, b, s, g1, g2, gate, scale, res, ds, dtype)
        check_backward(got, dn, b, s, g1, g2, gate, scale, res, ds, dtype, str(pair))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n", (1, 33, 1024, 4097, 20001))
def test_unusual_rows(n, dtype):
    """A constant row, a block of zeros, an empty stream, tiny and large rows, zero gradients, and
    gates and scales of zero."""
    rows = 8
    b, res, g1, g2 = operands(20, rows, n, dtype)
    dn, ds = make(21, rows, n, dtype), make(22, rows, n, dtype)
    b[0], b[1], res[2] = 3.0, 0.0, 0.0
    b[2] = 0.0
    b[3] = (b[3].float() * 1e-15).to(b.dtype)
    b[4] = (b[4].float() * 1e15).to(b.dtype)
    res[5] = (res[5].float() * 1e12).to(b.dtype)
    dn[6], ds[6] = 0.0, 0.0
    for pair in PAIRS:
        gate, scale = factors(8, rows, n, dtype, *pair)
        if gate is not None:
            gate.view(-1)[::3] = 0.0
        if scale is not None:
            scale.view(-1)[1::2] = 0.0
        s, y = run_forward(b, res, g1, g2, gate, scale, dtype)
        check_forward((s, y), b, res, g1, g2, gate, scale, dtype, str(pair))
        s = s.cpu()
        got = run_backward(dn, b, s, g1, g2, gate, scale, res, ds, dtype)
        check_backward(got, dn, b, s, g1, g2, gate, scale, res, ds, dtype, str(pair))
        assert not f64(got["dblock"])[6].any() and not f64(got["dresidual"])[6].any()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n", (7, 1024, 4097))
def test_streams_that_cancel(n, dtype):
    """The residual is the negative of the block's share but for a few percent: the second norm
    is of what is left."""
    rows = 300
    b, _, g1, g2 = operands(23, rows, n, dtype)
    gate, scale = factors(24, rows, n, dtype, "channel", "scalar")
    z, _ = gate_ref.stream(f64(b), np.zeros((rows, n)), f64(g1), f64(gate), f64(scale), E1)
    left = torch.randn(rows, n, generator=torch.Generator().manual_seed(25)).double() * 0.02
    res = ((left - torch.from_numpy(z)) / scale.double()).to(TYPES[dtype])
    got = run_forward(b, res, g1, g2, gate, scale, dtype)
    check_forward(got, b, res, g1, g2, gate, scale, dtype, "cancels")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n", (5, 1024, 4097))
def test_infinities_stay_in_their_rows(n, dtype):
    rows = 7
    b, res, g1, g2 = operands(30, rows, n, dtype)
    dn = make(31, rows, n, dtype)
    gate, _ = factors(32, rows, n, dtype, "row", "none")
    outs = []
    for poison in (False, True):
        b2, res2, dn2 = b.clone(), res.clone(), dn.clone()
        if poison:
            b2[2, n // 2] = float("nan")
            res2[4, n - 1] = float("inf")
            dn2[5, 0] = float("nan")
        s, y = run_forward(b2, res2, g1, g2, gate, None, dtype)
        got = run_backward(dn2, b2, s.cpu(), g1, g2, gate, None, None, None, dtype)
        outs.append([f64(t) for t in (s, y, got["dblock"], got["dresidual"], got["dgate"])])
    good = np.array([0, 1, 3, 6])
    for a, c in zip(*outs):
        assert np.array_equal(a[good], c[good])
    assert np.isnan(outs[1][1][[2, 4]]).any(1).all()
    assert np.isnan(outs[1][2][[2, 4, 5]]).any(1).all()


@pytest.mark.parametrize("rows,n", [(9, 40), (700, 512), (5, 4096), (320, 4095), (7, 140001)])
def test_an_infinite_scalar_gradient_is_infinite(rows, n):
    """One infinite incoming gradient makes the sums over all elements infinite, of its sign, where
    the formula's other terms are finite."""
    b, _, g1, g2 = (t.cuda() for t in operands(33, rows, n, "f32"))
    s, res, ds = make(34, rows, n, "f32").cuda(), make(35, rows, n, "f32").cuda(), torch.zeros(rows, n, device="cuda")
    one = torch.ones(1, device="cuda")
    for sign in (1.0, -1.0):
        ds[rows // 2, n // 3] = sign * float("inf")
        got = mrn.norm_gate_residual_norm_backward(torch.zeros_like(b), b, s, g1, g2, one, one,
                                                   residual=res, dstream=ds)
        at = rows // 2, n // 3
        assert float(got[5]) == sign * float("inf") * float(res[at].sign())
        assert float(got[4]) == sign * float("inf") * float((b[at] * g1[at[1]]).sign())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,n", [(5, 33), (40, 1023), (700, 512), (3, 20001), (1501, 1023),
                                    (2000, 99), (7, 140001)])
def test_in_place(rows, n, dtype):
    """Every output that may be one of the row inputs gives the bits it gives elsewhere."""
    b, res, g1, g2 = (t.cuda() for t in operands(40, rows, n, dtype))
    gate, scale = (t.cuda() for t in factors(41, rows, n, dtype, "row", "channel"))
    want = mrn.norm_gate_residual_norm(b, res, g1, g2, gate, scale)
    for k in range(2):
        v = [b.clone(), res.clone()]
        got = mrn.norm_gate_residual_norm(v[0], v[1], g1, g2, gate, scale, out_stream=v[k],
                                          normed=v[1 - k])
        assert got[0] is v[k] and all(torch.equal(p, q) for p, q in zip(got, want)), k
    s = want[0]
    dn, ds = make(42, rows, n, dtype).cuda(), make(43, rows, n, dtype).cuda()
    want = mrn.norm_gate_residual_norm_backward(dn, b, s, g1, g2, gate, scale, residual=res,
                                                dstream=ds)
    for k in range(5):
        v = [t.clone() for t in (dn, b, s, res, ds)]
        got = mrn.norm_gate_residual_norm_backward(
            v[0], v[1], v[2], g1, g2, gate, scale, residual=v[3], dstream=v[4], dblock=v[k],
            dresidual=v[(k + 1) % 5])
        assert all(torch.equal(p, q) for p, q in zip(got, want)), k


@pytest.mark.parametrize("dtype", DTYPES)
def test_operands_at_different_offsets(dtype):
    rows, n = 37, 1000
    t = TYPES[dtype]
    b, res, g1, g2 = operands(50, rows, n, dtype)
    dn, s = make(51, rows, n, dtype), make(52, rows, n, dtype)
    gate, scale = factors(53, rows, n, dtype, "channel", "channel")
    v = [Buf(tuple(x.shape), t, x, i).t for i, x in enumerate((b, res, g1, g2, gate, scale), 1)]
    o = [Buf((rows, n), t, None, i) for i in (3, 5)]
    got = mrn.norm_gate_residual_norm(*v, out_stream=o[0].t, normed=o[1].t)
    check_forward(got, b, res, g1, g2, gate, scale, dtype, "apart")
    got = mrn.norm_gate_residual_norm_backward(
        Buf((rows, n), t, dn, 2).t, v[0], Buf((rows, n), t, s, 3).t, v[2], v[3], v[4], v[5],
        residual=v[1], dblock=o[0].t, dresidual=o[1].t)
    assert all(x.guards_hold() for x in o)
    check_backward(dict(zip(OUTPUTS, got)), dn, b, s, g1, g2, gate, scale, res, None, dtype, "apart")
    # only the weights off their boundary, rows aligned
    got = mrn.norm_gate_residual_norm(b.cuda(), res.cuda(), *v[2:])
    check_forward(got, b, res, g1, g2, gate, scale, dtype, "weights apart")


def test_no_rows():
    n = 300
    x = torch.empty(0, n, device="cuda")
    g = torch.ones(n, device="cuda")
    nan = torch.full((n,), float("nan"), device="cuda")
    assert mrn.norm_gate_residual_norm(x, x, g, g, g, g)[1].shape == x.shape
    for gate, scale in ((g, g), (g[:1], g[:1]), (torch.empty(0, 1, device="cuda"), None)):
        got = mrn.norm_gate_residual_norm_backward(
            x, x, x, g, g, gate, scale, residual=x, dgamma_post=nan.clone(), dgamma_pre=nan.clone(),
            dgate=nan[:gate.numel()].clone().view(gate.shape),
            dres_scale=None if scale is None else nan[:scale.numel()].clone())
        for v in got[2:]:
            assert v is None or not v.any(), v


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,n", [(700, 513), (2000, 128), (400, 4096), (60, 20001)])
def test_same_call_same_bits(rows, n, dtype):
    """Twice in a row, on another stream and without programmatic launches."""
    b, res, g1, g2 = (t.cuda() for t in operands(60, rows, n, dtype))
    dn, ds = make(61, rows, n, dtype).cuda(), make(62, rows, n, dtype).cuda()
    gate, scale = (t.cuda() for t in factors(63, rows, n, dtype, "scalar", "scalar"))

    def step():
        s, y = mrn.norm_gate_residual_norm(b, res, g1, g2, gate, scale)
        return (s, y) + mrn.norm_gate_residual_norm_backward(dn, b, s, g1, g2, gate, scale,
                                                             residual=res, dstream=ds)

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
    for p, q, r in zip(first, second, third):
        assert torch.equal(p, q) and torch.equal(p, r)


def test_two_streams_at_once():
    """Calls that overlap in time, each with its own workspace."""
    rows, n = 3000, 1000
    streams = [torch.cuda.Stream() for _ in range(2)]
    b, dn, s = ([make(70 + 10 * k + i, rows, n, "bf16").cuda() for i in range(2)] for k in range(3))
    g = torch.ones(n, dtype=torch.bfloat16, device="cuda")
    gate = torch.full((1,), 0.5, dtype=torch.bfloat16, device="cuda")

    def call(i, **kw):
        return mrn.norm_gate_residual_norm_backward(dn[i], b[i], s[i], g, g, gate, **kw)[:5]

    want = [call(i) for i in range(2)]
    ws = [mrn.norm_gate_backward_workspace(b[i]) for i in range(2)]
    got = [None, None]
    torch.cuda.synchronize()
    for _ in range(20):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i] = call(i, workspace=ws[i])
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(p, q) for p, q in zip(got[i], want[i]))


def test_several_host_threads():
    """Calls of several threads, each on a stream of its own, give the bits of calls in turn."""
    rows, n = 400, 1000
    sets = []
    for i in range(4):
        b, res, g1, g2 = (t.cuda() for t in operands(110 + 10 * i, rows, n, "f32"))
        sets.append((b, res, g1, g2, *(t.cuda() for t in factors(i, rows, n, "f32", "scalar", "channel"))))

    def step(v):
        s, y = mrn.norm_gate_residual_norm(*v)
        grads = mrn.norm_gate_residual_norm_backward(y, v[0], s, v[2], v[3], v[4], v[5], residual=v[1])
        norm, grads = mrn.clip_grad_norm(grads, 0.5)
        return (s, y, norm, *grads)

    want = [step(v) for v in sets]
    torch.cuda.synchronize()
    got = [None] * len(sets)

    def run(i):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            for _ in range(10):
                got[i] = step(sets[i])
        stream.synchronize()

    threads = [threading.Thread(target=run, args=(i,)) for i in range(len(sets))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for a, c in zip(got, want):
        assert all(torch.equal(p, q) for p, q in zip(a, c))


def test_captured_tail_takes_the_factors_of_its_replay():
    rows, n = 90, 1023
    b, res, g1, g2 = (t.cuda() for t in operands(80, rows, n, "bf16"))
    gate, scale = (t.cuda() for t in factors(81, rows, n, "bf16", "row", "scalar"))
    dn = make(82, rows, n, "bf16").cuda()
    ws = mrn.norm_gate_backward_workspace(b)

    def step():
        s, y = mrn.norm_gate_residual_norm(b, res, g1, g2, gate, scale)
        return (s, y) + mrn.norm_gate_residual_norm_backward(dn, b, s, g1, g2, gate, scale,
                                                             residual=res, workspace=ws)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(3):
        gate.mul_(0.5)
        scale.add_(0.25)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        assert all(torch.equal(p, q) for p, q in zip(got, step())), i


FIRST_CALLS_CAPTURED = """
import torch
from dual_epsilon_sandwich_gb300 import mrn
b, res, dn = (torch.randn(40, 20001, device="cuda") for _ in range(3))
g1, g2, gate, scale = (torch.rand(20001, device="cuda") for _ in range(4))
ws, wl = mrn.norm_gate_backward_workspace(b), mrn.grad_norm_workspace([b, b])

def step():
    s, y = mrn.norm_gate_residual_norm(b, res, g1, g2, gate, scale)
    out = mrn.norm_gate_residual_norm_backward(dn, b, s, g1, g2, gate, scale, residual=res,
                                               workspace=ws)
    norm, out = mrn.clip_grad_norm(out[2:], 0.1, workspace=wl)
    return [t.clone() for t in (s, y, norm, *out)]

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


def test_helpers_refuse():
    x, g = torch.zeros(4, 8, device="cuda"), torch.ones(8, device="cuda")
    f, b = mrn.norm_gate_residual_norm, mrn.norm_gate_residual_norm_backward
    one, row = torch.ones(1, device="cuda"), torch.ones(4, 1, device="cuda")
    bad = [
        lambda: f(x.t(), x.t(), g, g), lambda: f(x, x, g[:4], g), lambda: f(x, x, g, g.bfloat16()),
        lambda: f(x, x[:2], g, g), lambda: f(x, x, g, g, gate=g.cpu()),
        lambda: f(x, x, g, g, gate=g[:3]), lambda: f(x, x, g, g, gate=g.bfloat16()),
        lambda: f(x, x, g, g, gate=row.view(4)), lambda: f(x, x, g, g, gate=one.view(())),
        lambda: f(x, x, g, g, res_scale=row), lambda: f(x, x, g, g, res_scale=x),
        lambda: f(x, x, g, g, eps_post=0.0), lambda: f(x, x, g, g, eps_pre=float("nan")),
        lambda: f(x, x, g, g, out_stream=x, normed=x), lambda: f(x, x, g, g, out_stream=x[0]),
        lambda: f(torch.zeros((), device="cuda"), x, g, g),
        lambda: b(x, x, x, g, g, dgate=one), lambda: b(x, x, x, g, g, one, dgate=g),
        lambda: b(x, x, x, g, g, one, one, dres_scale=one), lambda: b(x, x, x, g, g, one, dblock=x,
                                                                      dresidual=x),
        lambda: b(x, x, x, g, g, one, dgate=one.bfloat16()),
        lambda: b(x, x, x, g, g, residual=x[:2]), lambda: b(x, x, x, g, g, dstream=x.bfloat16()),
        lambda: b(x, x, x, g, g, dgamma_post=g.bfloat16()),
        lambda: b(x, x, x, g, g, workspace=torch.empty(4, dtype=torch.uint8, device="cuda")),
    ]
    for i, call in enumerate(bad):
        with pytest.raises((ValueError, TypeError, mrn.MrnError)):
            call()
            pytest.fail(f"call {i} was accepted")


class GatedTail(torch.autograd.Function):
    @staticmethod
    def forward(ctx, b, res, g1, g2, gate, scale):
        s, y = mrn.norm_gate_residual_norm(b, res, g1, g2, gate, scale)
        ctx.save_for_backward(b, s, g1, g2, gate, scale, res)
        return s, y

    @staticmethod
    def backward(ctx, ds, dn):
        db, dr, *rest = mrn.norm_gate_residual_norm_backward(
            dn.contiguous(), *ctx.saved_tensors, dstream=ds.contiguous())
        return db, dr, *rest


@pytest.mark.parametrize("kind", ("scalar", "channel", "row"))
def test_two_tails_a_loss_and_a_clip_against_autograd(kind):
    """A block's two tails forward and back, and its gradients clipped, as a training step runs
    them, against autograd in 64 bits."""
    rows, n, limit = 37, 1000, 0.5
    g = torch.Generator().manual_seed(95)
    b1, b2, r0, last = (torch.randn(rows, n, generator=g) for _ in range(4))
    w = [weights(96 + i, n, "f32")[0] for i in range(4)]
    f = [t for i in range(2) for t in factors(97 + i, rows, n, "f32", kind, "channel")]
    leaves = [t.cuda().requires_grad_() for t in (b1, b2, r0, *w, *f)]
    wide = [t.detach().double().cpu().requires_grad_() for t in leaves]

    def tail(b, r, g1, g2, gate, scale):
        s = scale * r + gate * (b / torch.sqrt((b * b).mean(1, keepdim=True) + E1) * g1)
        return s, s / torch.sqrt((s * s).mean(1, keepdim=True) + E2) * g2

    def step(tail, v):
        s, y = tail(v[0], v[2], v[3], v[4], v[7], v[8])
        s, y2 = tail(y + v[1], s, v[5], v[6], v[9], v[10])
        return y2 + 0.5 * s

    out, out64 = step(GatedTail.apply, leaves), step(tail, wide)
    got = torch.autograd.grad(out, leaves, last.cuda())
    want = torch.autograd.grad(out64, wide, last.double())
    # f32 all the way: a few hundred roundings of values of order one to ten
    for a, c in zip(got, want):
        assert float((a.cpu().double() - c).abs().max()) <= 512 * ref.U * float(c.abs().max())
    norm, clipped = mrn.clip_grad_norm(got, limit)
    total = torch.sqrt(sum((c * c).sum() for c in want))
    assert abs(float(norm) - float(total)) <= 512 * ref.U * float(total) and float(total) > limit
    for a, c in zip(clipped, want):
        c = c * (limit / total)
        assert float((a.cpu().double() - c).abs().max()) <= 1024 * ref.U * float(c.abs().max())


def test_a_gradient_is_not_lost_in_silence():
    x, g = torch.randn(4, 8, device="cuda"), torch.ones(8, device="cuda")
    t = {k: x.clone() for k in ("b", "res", "dn", "ds", "s", "o", "p")}
    t.update({k: g.clone() for k in ("g1", "g2", "gate", "scale", "d1", "d2", "d3", "d4")})
    calls = {
        "forward": (lambda: mrn.norm_gate_residual_norm(t["b"], t["res"], t["g1"], t["g2"], t["gate"],
                                                        t["scale"], out_stream=t["o"],
                                                        normed=t["p"]),
                    ("b", "res", "g1", "g2", "gate", "scale", "o", "p"), ("o", "p")),
        "backward": (lambda: mrn.norm_gate_residual_norm_backward(
            t["dn"], t["b"], t["s"], t["g1"], t["g2"], t["gate"], t["scale"], residual=t["res"],
            dstream=t["ds"], dblock=t["o"], dresidual=t["p"], dgamma_post=t["d1"],
            dgamma_pre=t["d2"], dgate=t["d3"], dres_scale=t["d4"]), tuple(t),
            ("o", "p", "d1", "d2", "d3", "d4"))}
    for name, (call, reads, writes) in calls.items():
        before = {k: v._version for k, v in t.items()}
        call()
        for k, v in t.items():
            assert (v._version > before[k]) == (k in writes), (name, k)
        for k in reads:
            t[k].requires_grad_()
            launches = mrn.mrn_launch_count()
            with pytest.raises(ValueError, match="requires a gradient"):
                call()
            assert mrn.mrn_launch_count() == launches, k
            with torch.no_grad():
                call()
            t[k].requires_grad_(False)


def test_past_32_bits():
    """More than 2^31 elements through the tail and its gradient: the last rows against the
    reference."""
    rows, n, last = 70001, 32771, 3
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB of device memory")
    gen = torch.Generator(device="cuda").manual_seed(98)
    b, res, dn = (torch.empty(rows, n, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
                  for _ in range(3))
    g1, g2 = weights(99, n, "bf16")[0], weights(100, n, "bf16")[0]
    gate, scale = factors(101, rows, n, "bf16", "row", "channel")
    s, y = mrn.norm_gate_residual_norm(b, res, g1.cuda(), g2.cuda(), gate.cuda(), scale.cuda())
    tail = [t[-last:].cpu() for t in (b, res, dn, s, y)]
    check_forward(tail[3:], tail[0], tail[1], g1, g2, gate[-last:], scale, "bf16", "last rows")
    got = mrn.norm_gate_residual_norm_backward(dn, b, s, g1.cuda(), g2.cuda(), gate.cuda(),
                                               scale.cuda(), dblock=y, dresidual=dn)
    want = gate_ref.backward(f64(tail[2]), f64(tail[0]), f64(tail[3]), f64(g1), f64(g2),
                             f64(gate[-last:]), f64(scale), None, E1, E2, None)
    for k, v in (("dblock", got[0]), ("dresidual", got[1]), ("dgate", got[4])):
        ref.check(f64(v[-last:]), *want[k], "f32" if k == "dgate" else "bf16", k)
def test_a_cluster_whose_messages_are_late_stops_and_recovers():
    """The test hook lets the first wait of a cluster expect bytes that never come: the calls
    return, mrn_wait_timeouts() reports them, and the next calls are exact."""
    rows, n = 3, 16384
    b, res, g1, g2 = operands(90, rows, n, "f32")
    s, dn = make(91, rows, n, "f32"), make(92, rows, n, "f32")
    v = [t.cuda() for t in (b, res, g1, g2, s, dn)]
    mrn.mrn_wait_timeouts()
    torch.cuda.synchronize()
    assert mrn.mrn_set_launch_options(mrn.MRN_LAUNCH_PDL | mrn.MRN_LAUNCH_TEST_WAIT_TIMEOUT) == 0
    try:
        t0 = time.perf_counter()
        mrn.norm_gate_residual_norm(*v[:4])
        mrn.norm_gate_residual_norm_backward(v[5], v[0], v[4], v[2], v[3])
        torch.cuda.synchronize()
        seconds = time.perf_counter() - t0
    finally:
        mrn.mrn_set_launch_options(mrn.MRN_LAUNCH_PDL)
    assert mrn.mrn_wait_timeouts() >= 2 and seconds < 30, seconds
    check_forward(run_forward(b, res, g1, g2, None, None, "f32"), b, res, g1, g2, None, None, "f32",
                  "after a timeout")
    got = run_backward(dn, b, s, g1, g2, None, None, None, None, "f32")
    check_backward(got, dn, b, s, g1, g2, None, None, None, None, "f32", "after a timeout")
    assert mrn.mrn_wait_timeouts() == 0


