"""The norm of many tensors and their clipping on the GPU against 64 bits."""
import math

import numpy as np
import pytest
import torch

import train_reference as ref
from dual_epsilon_sandwich_gb300 import mrn
from test_gpu_train import TYPES, Buf, f64

pytestmark = pytest.mark.gpu

# A thread adds at most 64 squares in one f32 chain (one more rounding each) before 64 bits take
# over: the sum of squares is off by 65 u, its root by 33, and the f32 it is stored in by one.
NORM = 34 * ref.U


@pytest.fixture(scope="module", autouse=True)
def library(gpu_lib):
    return gpu_lib


def tensors(seed, counts, dtypes, shifts, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return [Buf((c,), TYPES[d], (scale * torch.randn(c, generator=g)).to(TYPES[d]), s)
            for c, d, s in zip(counts, dtypes, shifts)]


def square(values):
    return math.fsum(float((f64(v) ** 2).sum()) for v in values)


def check_norm(norm, values, what=""):
    want = math.sqrt(square(values))
    assert abs(float(norm) - want) <= NORM * want + 1e-45, (what, float(norm), want)
    return want


def check_clip(norm, out, values, limit, what=""):
    want = check_norm(norm, values, what)
    k = min(1.0, limit / want) if want > 0.0 else 1.0
    for o, v in zip(out, values):
        v = f64(v)
        # the factor carries the norm's error and its own rounding, the product one of f32
        ref.check(f64(o), v * k, np.abs(v * k) * (NORM + 2 * ref.U),
                  "f32" if o.dtype == torch.float32 else "bf16", what)


LISTS = {
    "one element": ([1], ["f32"], [0]),
    "one small": ([7], ["bf16"], [3]),
    "empty ones": ([0, 5, 0, 0, 9, 0], ["f32", "bf16"] * 3, [0, 1, 2, 0, 1, 0]),
    "only empty": ([0, 0], ["f32", "bf16"], [0, 0]),
    "around vectors": ([3, 8, 15, 16, 17, 31, 33, 255, 256, 257], ["bf16", "f32"] * 5, range(10)),
    "around blocks": ([8191, 8192, 8193, 65537], ["f32", "bf16"] * 2, [0, 0, 5, 1]),
    "many tiny": ([1 + i % 5 for i in range(900)], ["bf16", "f32", "f32"] * 300, [0] * 900),
    "many": ([100 + 37 * i % 1000 for i in range(2500)], ["bf16"] * 1200 + ["f32"] * 1300,
             [i % 9 for i in range(2500)]),
    "large": ([3 << 20, 5, (1 << 22) + 13, 1 << 20], ["bf16", "f32", "f32", "bf16"], [0, 0, 1, 0]),
}


@pytest.mark.parametrize("name", LISTS)
def test_norm_and_clip(name):
    counts, dtypes, shifts = LISTS[name]
    bufs = tensors(1, counts, dtypes, list(shifts))
    values = [b.t.clone() for b in bufs]
    g = [b.t for b in bufs]
    ws = mrn.grad_norm_workspace(g)
    ws.view(torch.float64).fill_(float("nan"))     # nothing of it may be read before it is written
    want = check_norm(mrn.grad_norm(g, workspace=ws), values)
    for limit in (0.3 * want, 1.7 * want + 1.0, 0.0, float("inf")):
        outs = [Buf((c,), TYPES[d], None, s) for c, d, s in zip(counts, dtypes, shifts)]
        norm, out = mrn.clip_grad_norm(g, limit, out=[o.t for o in outs], workspace=ws)
        check_clip(norm, out, values, limit, f"limit {limit}")
        assert all(o.guards_hold() for o in outs)
        assert all(torch.equal(p, q) for p, q in zip(g, values))
        if limit > want:
            assert all(torch.equal(p, q) for p, q in zip(out, values))
    # in place, and at other offsets than the input's
    moved = [Buf((c,), TYPES[d], None, s + 1) for c, d, s in zip(counts, dtypes, shifts)]
    norm, out = mrn.clip_grad_norm(g, 0.3 * want, out=[o.t for o in moved], workspace=ws)
    check_clip(norm, out, values, 0.3 * want, "moved")
    assert all(o.guards_hold() for o in moved)
    again, same = mrn.clip_grad_norm(g, 0.3 * want, workspace=ws)
    assert same is g and torch.equal(again, norm)
    assert all(torch.equal(p, q) for p, q in zip(g, out)) and all(b.guards_hold() for b in bufs)


@pytest.mark.parametrize("count", (1, 50, 5000, 300000))
@pytest.mark.parametrize("dtype", ("f32", "bf16"))
@pytest.mark.parametrize("scale", (1e-38, 1e-30, 1e-20, 1e18, 1e25, 1e35))
def test_squares_that_leave_f32(scale, dtype, count):
    """The norm is right wherever it is an f32 number itself."""
    v = tensors(2, [count, 40], [dtype, "f32"], [0, 0], scale)
    g = [b.t for b in v]
    want = math.sqrt(square(g))
    norm = float(mrn.grad_norm(g))
    if want > 3.4e38:
        assert norm == float("inf")
        return
    # (subnormal inputs and a subnormal norm are exact to half of 2^-149)
    assert abs(norm - want) <= NORM * want + 1e-45
    _, out = mrn.clip_grad_norm(g, want / 4, out=[torch.empty_like(t) for t in g])
    for o, t in zip(out, g):
        ref.check(f64(o), f64(t) / 4, np.abs(f64(t)) * (NORM + 2 * ref.U) + 1e-40,
                  "f32" if t.dtype == torch.float32 else "bf16", "clip")


def test_large_beside_small():
    """Tensors whose squares lie far apart: each counts as far as it reaches."""
    g = [torch.full((5000,), v, device="cuda") for v in (1e-30, 1e-10, 1.0, 1e10)]
    check_norm(mrn.grad_norm(g[:1]), g[:1])
    check_norm(mrn.grad_norm(g[:2]), g[:2])
    check_norm(mrn.grad_norm(g), g)
    mixed = torch.full((70000,), 1e-25, device="cuda")
    mixed[::7] = 1e22
    check_norm(mrn.grad_norm([mixed]), [mixed])


@pytest.mark.parametrize("bad", (float("inf"), float("-inf"), float("nan")))
@pytest.mark.parametrize("at", (0, 9999, 123456))
def test_a_norm_that_is_not_finite_leaves_the_values(bad, at):
    g = [torch.randn(200000, device="cuda"), torch.randn(70, device="cuda").bfloat16()]
    g[0][at] = bad
    values = [t.clone() for t in g]
    assert str(float(mrn.grad_norm(g))) == str(abs(bad))
    norm, out = mrn.clip_grad_norm(g, 0.5, out=[torch.empty_like(t) for t in g])
    assert str(float(norm)) == str(abs(bad))
    mrn.clip_grad_norm(g, 0.5)
    for o, t, v in zip(out, g, values):
        w = v.view(torch.int16 if v.dtype == torch.bfloat16 else torch.int32)
        assert torch.equal(o.view(w.dtype), w) and torch.equal(t.view(w.dtype), w)


def test_listed_twice_counts_twice():
    t = torch.randn(1000, device="cuda")
    check_norm(mrn.grad_norm([t, t]), [t, t])
    out = [torch.empty_like(t) for _ in range(2)]
    mrn.clip_grad_norm([t, t], 1.0, out=out)
    assert torch.equal(out[0], out[1])


def test_same_call_same_bits():
    """Twice in a row, on another stream, without programmatic launches, and captured: a replay
    takes the values that it finds."""
    counts = [70001, 13, 4096, 1 << 18]
    g = [b.t for b in tensors(3, counts, ["bf16", "f32", "f32", "bf16"], [0, 1, 0, 0])]
    out = [torch.empty_like(t) for t in g]
    ws = mrn.grad_norm_workspace(g)

    def step():
        norm, _ = mrn.clip_grad_norm(g, 2.0, out=out, workspace=ws)
        return [t.clone() for t in (norm, *out)]

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
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    graph.replay()
    torch.cuda.synchronize()
    for p, *rest in zip(first, second, third, captured):
        assert all(torch.equal(p, q) for q in rest)
    for t in g:
        t.mul_(2)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(captured, step()))
    assert float(captured[0]) == 2 * float(first[0])


def test_helpers_refuse():
    x = torch.ones(16, device="cuda")
    y = torch.ones(16, device="cuda")
    bad = [
        lambda: mrn.grad_norm([x, x.cpu()]), lambda: mrn.grad_norm([x, x.half()]),
        lambda: mrn.grad_norm([x.view(4, 4).t()]), lambda: mrn.grad_norm([x], out=x[:2]),
        lambda: mrn.grad_norm([x], out=x[3]), lambda: mrn.grad_norm([x], out=y[:1].bfloat16()),
        lambda: mrn.grad_norm([x], workspace=torch.empty(8, dtype=torch.uint8, device="cuda")),
        lambda: mrn.grad_norm([x], workspace=y),
        lambda: mrn.clip_grad_norm([x, x], 1.0), lambda: mrn.clip_grad_norm([x[:9], x[8:]], 1.0),
        lambda: mrn.clip_grad_norm([x, y], 1.0, out=[y, x]),
        lambda: mrn.clip_grad_norm([x], 1.0, out=[y, y]),
        lambda: mrn.clip_grad_norm([x], 1.0, out=[y[:8]]),
        lambda: mrn.clip_grad_norm([x], 1.0, out=[y.bfloat16()]),
        lambda: mrn.clip_grad_norm([x], -1.0), lambda: mrn.clip_grad_norm([x], float("nan")),
        lambda: mrn.clip_grad_norm([x.clone().requires_grad_()], 1.0),
    ]
    for i, call in enumerate(bad):
        with pytest.raises((ValueError, TypeError, mrn.MrnError)):
            call()
            pytest.fail(f"call {i} was accepted")
    assert torch.equal(x, torch.ones_like(x)) and torch.equal(y, x)


def test_what_a_call_writes_counts_as_modified():
    x, y, n = torch.ones(16, device="cuda"), torch.ones(16, device="cuda"), torch.ones((), device="cuda")
    before = [t._version for t in (x, y, n)]
    mrn.grad_norm([x], out=n)
    mrn.clip_grad_norm([x], 1.0, out=[y], norm=n)
    assert x._version == before[0] and y._version > before[1] and n._version >= before[2] + 2
    mrn.clip_grad_norm([x], 1.0)
    assert x._version > before[0]


def test_past_32_bits():
    """A tensor of more than 2^32 elements: its last ones count, and are clipped."""
    count = (1 << 32) + 77
    if torch.cuda.mem_get_info()[0] < 20 << 30:
        pytest.skip("needs 20 GB of device memory")
    t = torch.zeros(count, dtype=torch.bfloat16, device="cuda")
    t[-1], t[-100], t[5], t[1 << 31] = 3.0, 4.0, 12.0, 84.0
    norm, _ = mrn.clip_grad_norm([t], 42.5)
    assert float(norm) == 85.0
    assert [float(t[i]) for i in (-1, -100, 5, 1 << 31)] == [1.5, 2.0, 6.0, 42.0]
    assert int((t != 0).sum()) == 4
