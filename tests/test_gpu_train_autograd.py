"""The training helpers beside autograd: what they return has no history, so that a tensor that
requires a gradient is refused while autograd records, and taken where it does not."""
import pytest
import torch

import train_reference as ref
from dual_epsilon_sandwich_gb300 import mrn

pytestmark = pytest.mark.gpu

ROWS, N, EPS, P = 9, 200, 1e-5, 0.25


@pytest.fixture(scope="module", autouse=True)
def library(gpu_lib):
    return gpu_lib


def operands():
    g = torch.Generator().manual_seed(5)
    t = {k: torch.randn(ROWS, N, generator=g).cuda()
         for k in ("x", "residual", "dy", "dstream", "out", "out2")}
    t.update({k: torch.randn(N, generator=g).cuda() for k in ("gamma", "beta", "dgamma", "dbeta")})
    t.update({k: torch.rand(ROWS, generator=g).cuda() + 0.5 for k in ("mean", "rstd")})
    t["rng"] = torch.tensor([3, 4], device="cuda")
    return t


# every helper with all its tensors, and the names of those that may require a gradient
CALLS = {
    "layernorm": (lambda t: mrn.layernorm(t["x"], t["gamma"], t["beta"], EPS, out=t["out"],
                                          mean=t["mean"], rstd=t["rstd"]),
                  ("x", "gamma", "beta", "out", "mean", "rstd")),
    "dropout_add": (lambda t: mrn.dropout_add(t["x"], t["residual"], P, t["rng"], out=t["out"]),
                    ("x", "residual", "out")),
    "dropout alone": (lambda t: mrn.dropout_add(t["x"], None, P, t["rng"]), ("x",)),
    "dropout_add_layernorm": (
        lambda t: mrn.dropout_add_layernorm(t["x"], t["residual"], t["gamma"], t["beta"], EPS, P,
                                            t["rng"], out_stream=t["out"], normed=t["out2"],
                                            mean=t["mean"], rstd=t["rstd"]),
        ("x", "residual", "gamma", "beta", "out", "out2", "mean", "rstd")),
    "layernorm_backward": (
        lambda t: mrn.layernorm_backward(t["dy"], t["x"], t["gamma"], t["mean"], t["rstd"],
                                         dstream=t["dstream"], dx=t["out"], dgamma=t["dgamma"],
                                         dbeta=t["dbeta"]),
        ("dy", "x", "gamma", "mean", "rstd", "dstream", "out", "dgamma", "dbeta")),
    "dropout_add_layernorm_backward": (
        lambda t: mrn.dropout_add_layernorm_backward(
            t["dy"], t["x"], t["gamma"], t["mean"], t["rstd"], P, t["rng"], dstream=t["dstream"],
            dx=t["out"], dresidual=t["out2"], dgamma=t["dgamma"], dbeta=t["dbeta"]),
        ("dy", "x", "gamma", "mean", "rstd", "dstream", "out", "out2", "dgamma", "dbeta")),
    "rmsnorm_backward": (
        lambda t: mrn.rmsnorm_backward(t["dy"], t["x"], t["gamma"], EPS, dstream=t["dstream"],
                                       dx=t["out"], dgamma=t["dgamma"]),
        ("dy", "x", "gamma", "dstream", "out", "dgamma")),
}


def flat(r):
    return [t.clone() for t in (r if isinstance(r, tuple) else (r,))]


@pytest.mark.parametrize("name", CALLS)
def test_a_gradient_is_not_lost_in_silence(name):
    call, names = CALLS[name]
    want = flat(call(operands()))
    for k in names:
        t = operands()
        t[k].requires_grad_()
        before = mrn.mrn_launch_count()
        with pytest.raises(ValueError, match="requires a gradient"):
            call(t)
        assert mrn.mrn_launch_count() == before, k
        with torch.no_grad():
            got = flat(call(t))
        assert all(torch.equal(a, b) for a, b in zip(got, want)), k
    x = operands()["x"].requires_grad_()
    assert mrn.norm_backward_workspace(x).numel() > 0        # (loses nothing)


class LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, gamma, beta):
        mean, rstd = torch.empty(len(x), device=x.device), torch.empty(len(x), device=x.device)
        y = mrn.layernorm(x, gamma, beta, EPS, mean=mean, rstd=rstd)
        ctx.save_for_backward(x, gamma, mean, rstd)
        return y

    @staticmethod
    def backward(ctx, dy):
        return mrn.layernorm_backward(dy, *ctx.saved_tensors)


def test_from_an_autograd_function():
    """The gradients of autograd in 64 bits; a second derivative, which the helpers do not
    have, is refused."""
    t = operands()
    leaves = [t[k].requires_grad_() for k in ("x", "gamma", "beta")]
    y = LayerNorm.apply(*leaves)
    got = torch.autograd.grad(y, leaves, t["dy"], retain_graph=True)
    x, g, b = (v.detach().double().requires_grad_() for v in leaves)
    d = x - x.mean(1, keepdim=True)
    y64 = d / (d.square().mean(1, keepdim=True) + EPS).sqrt() * g + b
    want = torch.autograd.grad(y64, (x, g, b), t["dy"].double())
    for u, v in zip((y.detach(), *got), (y64.detach(), *want)):
        # a few hundred roundings of values of order one to ten
        assert float((u.double() - v).abs().max()) <= 512 * ref.U * float(v.abs().max())
    with pytest.raises(ValueError, match="requires a gradient"):
        torch.autograd.grad(y, leaves, t["dy"].requires_grad_(), create_graph=True)


WRITTEN = {"layernorm": ("out", "mean", "rstd"), "dropout_add": ("out",),
           "dropout_add_layernorm": ("out", "out2", "mean", "rstd"),
           "layernorm_backward": ("out", "dgamma", "dbeta"),
           "dropout_add_layernorm_backward": ("out", "out2", "dgamma", "dbeta"),
           "rmsnorm_backward": ("out", "dgamma")}


@pytest.mark.parametrize("name", WRITTEN)
def test_what_a_call_writes_counts_as_modified(name):
    """... and what it reads does not; tensors of inference mode, which have no count, are taken."""
    call, _ = CALLS[name]
    t = operands()
    before = {k: v._version for k, v in t.items()}
    call(t)
    for k, v in t.items():
        assert (v._version > before[k]) == (k in WRITTEN[name]), k
    with torch.inference_mode():
        want = flat(call(operands()))
    assert all(torch.equal(a, b) for a, b in zip(flat(call(operands())), want))


def test_autograd_notices_a_call_in_place():
    """exp keeps its result for its gradient; a call that overwrites it makes the gradient an
    error, as torch's own operations in place do."""
    t = operands()
    leaf = t["x"].requires_grad_()
    for write in (lambda v: mrn.layernorm(v, t["gamma"], t["beta"], EPS, out=v),
                  lambda v: mrn.dropout_add(v, t["residual"], P, t["rng"], out=v),
                  lambda v: mrn.rmsnorm_backward(t["dy"], v, t["gamma"], EPS, dx=v)):
        y = leaf.exp()
        with torch.no_grad():
            write(y)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            y.sum().backward()
