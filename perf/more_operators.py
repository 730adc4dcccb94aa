"""The gated sandwich tail with its gradient, and the global gradient norm with clipping,
measured: the tail of a sub-block between its two norms where the block has a gate and the
stream a residual scale, and what ends a training step's backward pass.

``listed()`` and ``draw()`` give cases, ``prepare()`` what a program holds before a call,
``run()`` one pass through one operator: in plain torch where ``own`` is false, through
``dual_epsilon_sandwich_gb300.mrn`` where it is true.  ``exact()`` is the definition in 64
bits.  All of them are bound by memory: ``work()`` counts each input read once and each
output written once.

Formulas (row r of a [rows x n] matrix, j = 0 .. n-1; inv(v; e) = 1 / sqrt(sum_j v_j^2 / n + e)):

  norm_gate_residual_norm
      xh = block_out * inv(block_out; eps_post)
      out_stream = res_scale * residual + gate * gamma_post * xh, rounded once and stored
      normed = out_stream * inv(out_stream; eps_pre) * gamma_pre
    gate: none (one), a scalar, one value per channel (j) or one per row (r);
    res_scale: none (one), a scalar or one value per channel
  norm_gate_residual_norm_backward, from dnormed and dstream (the stream's own gradient)
      i = inv(out_stream; eps_pre), w = dnormed * gamma_pre
      ds = i * (w - out_stream * i^2 * sum_j (w * out_stream) / n) [+ dstream]
      u = ds * gate * gamma_post
      dblock = inv(block_out; eps_post) * (u - xh * sum_j (u * xh) / n)
      dresidual = res_scale * ds
      dgamma_pre = sum_r dnormed * out_stream * i,  dgamma_post = sum_r ds * gate * xh
      dgate = ds * gamma_post * xh and dres_scale = ds * residual, summed over what shares a value
  grad_norm        norm = sqrt(sum over tensors and elements of g^2)
  clip_grad_norm   norm, and g * min(1, max_norm / norm) for every tensor
"""
import math

import torch

own = False

_TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
_TAILS = ("norm_gate_residual_norm", "norm_gate_residual_norm_backward")
_LISTS = ("grad_norm", "clip_grad_norm")


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def listed():
    def tail(name, op, dtype, rows, n, gate, scale, **more):
        c = {"name": name, "op": op, "dtype": dtype, "rows": rows, "n": n, "gate": gate,
             "scale": scale, "eps_post": 1e-8, "eps_pre": 1e-5, "dstream": True}
        c.update(more)
        return c

    def grads(name, op, dtype, width, inner, vocab, layers, clip=0.25):
        return {"name": name, "op": op, "dtype": dtype, "width": width, "inner": inner,
                "vocab": vocab, "layers": layers, "odd": 0, "clip": clip}

    fwd, bwd = _TAILS
    norm, clip = _LISTS
    return [
        # one token through a sub-block's tail, a learned gate per channel: latency counts
        tail("gate_f32_1x6656", fwd, "f32", 1, 6656, "channel", "scalar"),
        # a long prompt or a training batch, the same gate
        tail("gate_bf16_16384x4096", fwd, "bf16", 16384, 4096, "channel", "scalar"),
        # a gate per token, rows whose pitch is not a multiple of 16 bytes
        tail("gate_f32_4096x6655", fwd, "f32", 4096, 6655, "row", "none"),
        # a micro-batch of a small model, scalar gate and scale: latency counts
        tail("gate_grad_f32_64x768", bwd, "f32", 64, 768, "scalar", "scalar", dstream=False),
        # a training batch, gate and residual scale learned per channel
        tail("gate_grad_bf16_16384x4096", bwd, "bf16", 16384, 4096, "channel", "channel"),
        # the same rows an element narrower, a gate per token
        tail("gate_grad_bf16_16384x4095", bwd, "bf16", 16384, 4095, "row", "none"),
        # the sandwich tail's own gradient (no gate) at the pages' model width
        tail("gate_grad_f32_4096x6656", bwd, "f32", 4096, 6656, "none", "none"),
        # the gradients of the norms' weights alone, 2 x 52 layers of the pages' model: many
        # small tensors, latency counts
        grads("norm_f32_104_weights", norm, "f32", 6656, 0, 0, 52),
        # every gradient of a model of 0.6 G parameters
        grads("norm_bf16_0.6G", norm, "bf16", 2048, 5632, 32000, 10),
        # one layer's gradients
        grads("clip_f32_1_layer", clip, "f32", 1024, 4096, 0, 1),
        # matrices in bf16 beside norm weights in f32, whose norm the limit does not reach
        grads("clip_mixed_0.2G", clip, "mixed", 1024, 2816, 32000, 11, clip=2.0),
        # every gradient of a model of 0.6 G parameters
        grads("clip_bf16_0.6G", clip, "bf16", 2048, 5632, 32000, 10),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    """One more case.  Tails: widths 32 .. 16384 and rows 1 .. 65536 over their logarithm (2^26
    elements at most), half of the widths multiples of 32, the others any number.  Lists: widths
    32 .. 4096, up to 24 layers and 0.5 G elements, a few tensors of odd sizes beside them."""
    if rng.random() < 0.6:
        n = _log(rng, 32, 16384)
        if rng.random() < 0.5:
            n = max(32, n // 32 * 32)
        rows = _log(rng, 1, min(65536, (1 << 26) // n))
        return {"op": rng.choice(_TAILS), "dtype": rng.choice(("f32", "bf16")), "rows": rows,
                "n": n, "gate": rng.choice(("none", "scalar", "channel", "row")),
                "scale": rng.choice(("none", "scalar", "channel")),
                "eps_post": rng.choice((1e-5, 1e-6, 1e-8)),
                "eps_pre": rng.choice((1e-5, 1e-6)), "dstream": rng.random() < 0.5}
    while True:
        c = {"op": rng.choice(_LISTS), "dtype": rng.choice(("f32", "bf16", "mixed")),
             "width": _log(rng, 32, 4096), "inner": rng.choice((0, _log(rng, 64, 8192))),
             "vocab": rng.choice((0, _log(rng, 256, 32000))), "layers": rng.randint(1, 24),
             "odd": rng.randint(0, 5), "clip": rng.choice((0.05, 0.25, 0.9, 1.5))}
        if sum(math.prod(s) for s, _ in _tensors(c)) <= 1 << 29:
            return c


def _tensors(c):
    """(shape, type) of every gradient of a list case, in a model's order: the embedding, per
    layer a norm, query, key, value and output, a norm, the inner block's three matrices, and
    then tensors of odd sizes, one of them empty."""
    d, m = c["width"], c["inner"]
    big = torch.float32 if c["dtype"] == "f32" else torch.bfloat16
    small = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
    out = [((c["vocab"], d), big)] if c["vocab"] else []
    for _ in range(c["layers"]):
        out.append(((d,), small))
        if m:
            out += [((d, d), big)] * 4
        out.append(((d,), small))
        if m:
            out += [((m, d), big), ((m, d), big), ((d, m), big)]
    for i in range(c["odd"]):
        out.append((((1, 0, d + 1, 31 * d + 7, 5)[i],), (small, big)[i % 2]))
    return out


def prepare(case, seed):
    """Inputs on the GPU.  The block's output is N(0, 1) with a scale per row log-uniform over
    0.01 .. 100, the stream's rows N(0, 1), weights 1 + 0.1 N(0, 1), gates per channel 0.1
    + 0.1 N(0, 1), gates per row between 0 and 1, incoming gradients N(0, 1).  Gradients of a
    list are normal with a deviation of each tensor's own, 10^-4 .. 10^-1."""
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    s = {"case": case}
    if case["op"] in _LISTS:
        return _prepare_list(case, s, g, dev)
    rows, n, t = case["rows"], case["n"], _TYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    scale = 10.0 ** (4.0 * torch.rand(rows, 1, generator=g, device=dev) - 2.0)
    s["block_out"] = (normal(rows, n) * scale).to(t)
    s["residual"] = normal(rows, n).to(t)
    s["gamma_post"] = (1.0 + 0.1 * normal(n)).to(t)
    s["gamma_pre"] = (1.0 + 0.1 * normal(n)).to(t)
    gates = {"none": lambda: None,
             "scalar": lambda: (0.5 + 0.1 * normal(1)).to(t),
             "channel": lambda: (0.1 + 0.1 * normal(n)).to(t),
             "row": lambda: torch.rand(rows, 1, generator=g, device=dev).to(t)}
    s["gate"] = gates[case["gate"]]()
    scales = {"none": lambda: None, "scalar": lambda: (0.9 + 0.1 * normal(1)).to(t),
              "channel": lambda: (1.0 + 0.1 * normal(n)).to(t)}
    s["res_scale"] = scales[case["scale"]]()
    # the buffers that a program keeps from step to step
    if case["op"] == _TAILS[0]:
        s["out"] = {"out_stream": torch.empty_like(s["residual"]),
                    "normed": torch.empty_like(s["residual"])}
        return s
    s["out_stream"] = _tail_plain(s)[0]
    s["dnormed"] = normal(rows, n).to(t)
    s["dstream"] = normal(rows, n).to(t) if case["dstream"] else None
    s["out"] = {"dblock": torch.empty_like(s["residual"]),
                "dresidual": torch.empty_like(s["residual"]),
                "dgamma_post": torch.empty(n, device=dev),
                "dgamma_pre": torch.empty(n, device=dev)}
    if s["gate"] is not None:
        s["out"]["dgate"] = torch.empty(s["gate"].shape, device=dev)
    if s["res_scale"] is not None:
        s["out"]["dres_scale"] = torch.empty(s["res_scale"].shape, device=dev)
    else:
        s["residual"] = None                       # (the gradient does not need it)
    if own:
        from dual_epsilon_sandwich_gb300 import mrn
        s["workspace"] = mrn.norm_gate_backward_workspace(s["block_out"])
    return s


def _views(flat, shapes):
    """The list's tensors as views of one buffer per type, one behind the other."""
    at = dict.fromkeys(flat, 0)
    out = []
    for shape, t in shapes:
        count = math.prod(shape)
        out.append(flat[t][at[t]:at[t] + count].view(shape))
        at[t] += count
    return out


def _prepare_list(case, s, g, dev):
    shapes = _tensors(case)
    sigma = 10.0 ** (3.0 * torch.rand(len(shapes), generator=g, device=dev) - 4.0)
    if case["op"] == "clip_grad_norm":
        # flat gradients, one buffer per type, as data parallel training keeps them
        size = {}
        for shape, t in shapes:
            size[t] = size.get(t, 0) + math.prod(shape)
        s["flat"] = {t: torch.empty(v, dtype=t, device=dev) for t, v in size.items()}
        s["flat_out"] = {t: torch.empty_like(v) for t, v in s["flat"].items()}
        s["grads"], s["out"] = _views(s["flat"], shapes), _views(s["flat_out"], shapes)
    else:
        s["grads"] = [torch.empty(shape, dtype=t, device=dev) for shape, t in shapes]
    for i, v in enumerate(s["grads"]):
        v.normal_(generator=g).mul_(sigma[i].to(v.dtype))
    square = sum(math.prod(shape) * d * d for (shape, _), d in zip(shapes, sigma.tolist()))
    s["max_norm"] = case["clip"] * math.sqrt(square)
    s["norm"] = torch.empty((), device=dev)
    if own:
        from dual_epsilon_sandwich_gb300 import mrn
        s["workspace"] = mrn.grad_norm_workspace(s["grads"])
    return s


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------
def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(s):
    from dual_epsilon_sandwich_gb300 import mrn
    c = s["case"]
    if c["op"] == "grad_norm":
        return {"norm": mrn.grad_norm(s["grads"], out=s["norm"], workspace=s["workspace"])}
    if c["op"] == "clip_grad_norm":
        norm, _ = mrn.clip_grad_norm(s["grads"], s["max_norm"], out=s["out"], norm=s["norm"],
                                     workspace=s["workspace"])
        return _clipped(norm, s["flat_out"])
    o = s["out"]
    if c["op"] == _TAILS[0]:
        mrn.norm_gate_residual_norm(s["block_out"], s["residual"], s["gamma_post"],
                                    s["gamma_pre"], gate=s["gate"], res_scale=s["res_scale"],
                                    eps_post=c["eps_post"], eps_pre=c["eps_pre"],
                                    out_stream=o["out_stream"], normed=o["normed"])
    else:
        mrn.norm_gate_residual_norm_backward(
            s["dnormed"], s["block_out"], s["out_stream"], s["gamma_post"], s["gamma_pre"],
            gate=s["gate"], res_scale=s["res_scale"], residual=s["residual"],
            eps_post=c["eps_post"], eps_pre=c["eps_pre"], dstream=s["dstream"],
            dblock=o["dblock"], dresidual=o["dresidual"], dgamma_post=o["dgamma_post"],
            dgamma_pre=o["dgamma_pre"], dgate=o.get("dgate"), dres_scale=o.get("dres_scale"),
            workspace=s["workspace"])
    return dict(o)


def _clipped(norm, flat):
    """The norm and every gradient, in the flat buffers that hold them."""
    out = {"norm": norm}
    out.update(("f32" if t == torch.float32 else "bf16", v) for t, v in flat.items())
    return out


def _f32(v):
    return 1.0 if v is None else v.float()


def _inv(v, eps):
    return 1.0 / torch.sqrt((v * v).sum(-1, keepdim=True) / v.shape[-1] + eps)


def _tail_plain(s):
    c = s["case"]
    t = _TYPES[c["dtype"]]
    b = s["block_out"].float()
    z = b * _inv(b, c["eps_post"]) * s["gamma_post"].float() * _f32(s["gate"])
    stream = (_f32(s["res_scale"]) * s["residual"].float() + z).to(t)
    v = stream.float()
    return stream, (v * _inv(v, c["eps_pre"]) * s["gamma_pre"].float()).to(t)


def _shared(per_element, like):
    """Sums per_element over what shares a value of `like`."""
    if like.numel() == 1:
        return per_element.sum().reshape(like.shape)
    if like.dim() == 2:
        return per_element.sum(-1, keepdim=True)
    return per_element.sum(0)


def _tail_backward_plain(s):
    c = s["case"]
    n, t = c["n"], _TYPES[c["dtype"]]
    v, dn = s["out_stream"].float(), s["dnormed"].float()
    i = _inv(v, c["eps_pre"])
    vh = v * i
    w = dn * s["gamma_pre"].float()
    ds = i * (w - vh * ((w * vh).sum(-1, keepdim=True) / n))
    if s["dstream"] is not None:
        ds = ds + s["dstream"].float()
    b = s["block_out"].float()
    i = _inv(b, c["eps_post"])
    xh = b * i
    gate, gamma = _f32(s["gate"]), s["gamma_post"].float()
    u = ds * gate * gamma
    db = i * (u - xh * ((u * xh).sum(-1, keepdim=True) / n))
    out = {"dblock": db.to(t), "dresidual": (_f32(s["res_scale"]) * ds).to(t),
           "dgamma_post": (ds * gate * xh).sum(0), "dgamma_pre": (dn * vh).sum(0)}
    if s["gate"] is not None:
        out["dgate"] = _shared(ds * gamma * xh, s["gate"])
    if s["res_scale"] is not None:
        out["dres_scale"] = _shared(ds * s["residual"].float(), s["res_scale"])
    return out


def _run_plain(s):
    op = s["case"]["op"]
    if op == _TAILS[0]:
        stream, normed = _tail_plain(s)
        return {"out_stream": stream, "normed": normed}
    if op == _TAILS[1]:
        return _tail_backward_plain(s)
    square = torch.zeros((), dtype=torch.float64, device="cuda")
    for v in s["grads"]:                             # (64 bits: a sum over all parameters)
        f = v.float()
        square += (f * f).sum(dtype=torch.float64)
    norm = torch.sqrt(square)
    if op == "grad_norm":
        return {"norm": norm.float()}
    coef = torch.clamp(s["max_norm"] / norm, max=1.0).float()
    for v, o in zip(s["grads"], s["out"]):
        o.copy_((v.float() * coef).to(v.dtype))
    return _clipped(norm.float(), s["flat_out"])


# ---------------------------------------------------------------------------
# The definition in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in _LISTS:
        norm = math.sqrt(math.fsum(float(v.double().square().sum()) for v in s["grads"]))
        at = torch.tensor(norm, dtype=torch.float64, device="cuda")
        if case["op"] == "grad_norm":
            return {"norm": at}
        coef = min(1.0, s["max_norm"] / norm) if norm > 0.0 else 1.0
        return _clipped(at, {t: v.double() * coef for t, v in s["flat"].items()})

    def wide(v, otherwise=None):
        return otherwise if v is None else v.double()

    one = torch.ones((), dtype=torch.float64, device="cuda")
    b, gamma, gamma2 = (wide(s[k]) for k in ("block_out", "gamma_post", "gamma_pre"))
    gate, scale = wide(s["gate"], one), wide(s["res_scale"], one)
    r1 = (b.square().mean(-1, keepdim=True) + case["eps_post"]).rsqrt()
    xh = b * r1
    if case["op"] == _TAILS[0]:
        stream = scale * wide(s["residual"]) + gate * gamma * xh
        v = stream.to(_TYPES[case["dtype"]]).double()
        r2 = (v.square().mean(-1, keepdim=True) + case["eps_pre"]).rsqrt()
        return {"out_stream": stream, "normed": v * r2 * gamma2}
    v, dn = wide(s["out_stream"]), wide(s["dnormed"])
    r2 = (v.square().mean(-1, keepdim=True) + case["eps_pre"]).rsqrt()
    vh = v * r2
    w = dn * gamma2
    ds = r2 * (w - vh * (w * vh).mean(-1, keepdim=True))
    if s["dstream"] is not None:
        ds += wide(s["dstream"])
    u = ds * (gate * gamma)
    out = {"dblock": r1 * (u - xh * (u * xh).mean(-1, keepdim=True)), "dresidual": scale * ds,
           "dgamma_post": (ds * xh * gate).sum(0), "dgamma_pre": (dn * vh).sum(0)}
    axes = {"scalar": (0, 1), "channel": (0,), "row": (1,)}
    if case["gate"] != "none":
        out["dgate"] = (ds * gamma * xh).sum(axes[case["gate"]]).reshape(s["gate"].shape)
    if case["scale"] != "none":
        out["dres_scale"] = (ds * wide(s["residual"])).sum(axes[case["scale"]]).reshape(
            s["res_scale"].shape)
    return out


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    if case["op"] in _LISTS:
        tensors = _tensors(case)
        count = sum(math.prod(s) for s, _ in tensors)
        size = sum(math.prod(s) * (4 if t == torch.float32 else 2) for s, t in tensors)
        if case["op"] == "grad_norm":
            return {"bytes": size + 4, "flops": 2 * count}
        return {"bytes": 2 * size + 4, "flops": 3 * count}
    rows, n = case["rows"], case["n"]
    size = 4 if case["dtype"] == "f32" else 2
    shared = {"none": 0, "scalar": 1, "channel": n, "row": rows}
    weights = 2 * n + shared[case["gate"]] + shared[case["scale"]]
    if case["op"] == _TAILS[0]:
        return {"bytes": (4 * rows * n + weights) * size, "flops": 11 * rows * n}
    matrices, flops = 5, 26                  # dnormed, block_out, out_stream; dblock, dresidual
    if case["dstream"]:
        matrices, flops = matrices + 1, flops + 1
    sums = 2 * n + shared[case["gate"]] + shared[case["scale"]]
    if case["scale"] != "none":
        matrices, flops = matrices + 1, flops + 3
    return {"bytes": (matrices * rows * n + weights) * size + 4 * sums, "flops": flops * rows * n}
