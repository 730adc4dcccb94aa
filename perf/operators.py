"""The training operators of the norms, measured: LayerNorm and its gradient,
the residual add with dropout (alone and before a LayerNorm) and its gradient,
and the gradient of RMSNorm.

``listed()`` and ``draw()`` give cases, ``prepare()`` what a program holds
before a call, ``run()`` one pass through one operator: in plain torch where
``own`` is false, through ``dual_epsilon_sandwich_gb300.mrn`` where it is true.
``exact()`` is the definition in 64 bits.  All of them are bound by memory:
``work()`` counts each input read once and each output written once.

Formulas (row r of a [rows x n] matrix, j = 0 .. n-1, e = r*n + j):

  layernorm        y = (x - mean) * rstd * gamma + beta,
                   mean = sum_j x / n, rstd = 1 / sqrt(sum_j (x - mean)^2 / n + eps)
  its gradient     xh = (x - mean) * rstd, w = dy * gamma,
                   dx = rstd * (w - sum_j w / n - xh * sum_j (w * xh) / n) [+ dstream],
                   dgamma = sum_r dy * xh, dbeta = sum_r dy
  rmsnorm gradient inv = 1 / sqrt(sum_j x^2 / n + eps), w = dy * gamma,
                   dx = inv * (w - x * inv^2 * sum_j (w * x) / n) [+ dstream],
                   dgamma = sum_r dy * x * inv
  dropout          keep(e) = u16(e) >= t, t = round(p * 2^16), and kept values are
                   multiplied by 2^16 / (2^16 - t); u16(e) is lane e % 8 (16 bits, low
                   half of each word first) of Philox4x32-10 (Salmon, Moraes, Dror, Shaw,
                   "Parallel random numbers: as easy as 1, 2, 3", 2011) with the counter
                   (e / 8, rng[1] + site), 64 bits each, and the key rng[0]
  dropout_add      out = residual + dropout(x)
  dropout_add_layernorm           s = residual + dropout(x), rounded once to the operands'
                                  type and stored; normed = layernorm(s)
  dropout_add_layernorm_backward  ds = layernorm gradient of dnormed at s, + dstream;
                                  dresidual = ds, dx = dropout(ds), dgamma, dbeta
"""
import math

import torch

own = False

_TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def listed():
    def case(name, op, dtype, rows, n, **more):
        c = {"name": name, "op": op, "dtype": dtype, "rows": rows, "n": n, "eps": 1e-5,
             "bias": True, "p": 0.1, "dstream": True}
        c.update(more)
        return c

    return [
        # a few rows through a LayerNorm, as at evaluation: latency counts
        case("layernorm_f32_4x6656", "layernorm", "f32", 4, 6656),
        # a training batch's LayerNorm, statistics kept for its gradient
        case("layernorm_bf16_16384x4096", "layernorm", "bf16", 16384, 4096),
        # a micro-batch's residual add with dropout: latency counts
        case("drop_add_bf16_64x2048", "dropout_add", "bf16", 64, 2048),
        # the residual add of a large batch, two gigabytes in and out
        case("drop_add_bf16_65536x5120", "dropout_add", "bf16", 65536, 5120),
        # rows whose pitch is not a multiple of 16 bytes
        case("drop_add_ln_f32_4096x6655", "dropout_add_layernorm", "f32", 4096, 6655),
        # the tail of a training sub-block: dropout, residual add, the next norm
        case("drop_add_ln_bf16_16384x4096", "dropout_add_layernorm", "bf16", 16384,
             4096),
        # the gradient of a small model's or micro-batch's norm: latency counts
        case("layernorm_grad_f32_64x768", "layernorm_backward", "f32", 64, 768,
             dstream=False),
        # the gradient of a training batch's norm
        case("layernorm_grad_bf16_16384x4096", "layernorm_backward", "bf16", 16384, 4096,
             dstream=False),
        # the gradient of the training sub-block's tail, odd width
        case("drop_add_ln_grad_bf16_16384x4095", "dropout_add_layernorm_backward",
             "bf16", 16384, 4095),
        # the same at the pages' model width in f32
        case("drop_add_ln_grad_f32_4096x6656", "dropout_add_layernorm_backward",
             "f32", 4096, 6656),
        # the gradient of the per-head norm of queries and keys: many short rows
        case("rmsnorm_grad_bf16_163840x128", "rmsnorm_backward", "bf16", 163840, 128,
             dstream=False),
        # the gradient of a pre norm of wide rows, the stream's own gradient added
        case("rmsnorm_grad_f32_4096x16384", "rmsnorm_backward", "f32", 4096, 16384),
    ]


_OPS = ("layernorm", "dropout_add", "dropout_add_layernorm", "layernorm_backward",
        "dropout_add_layernorm_backward", "rmsnorm_backward")


def draw(rng):
    """One more case: widths 32 .. 16384 and rows 1 .. 65536 over their logarithm (2^26
    elements at most), half of the widths multiples of 32, the others any number."""
    n = int(round(math.exp(rng.uniform(math.log(32), math.log(16384)))))
    if rng.random() < 0.5:
        n = max(32, n // 32 * 32)
    top = min(65536, (1 << 26) // n)
    rows = max(1, int(round(math.exp(rng.uniform(0.0, math.log(top))))))
    return {"op": rng.choice(_OPS), "dtype": rng.choice(("f32", "bf16")), "rows": rows, "n": n,
            "eps": rng.choice((1e-5, 1e-6, 1e-8)), "bias": rng.random() < 0.75,
            "p": rng.choice((0.0, 0.05, 0.1, 0.25, 0.5)), "dstream": rng.random() < 0.5}


def prepare(case, seed):
    """Inputs on the GPU.  Rows have a mean of their own and a scale log-uniform over
    0.01 .. 100 (layernorm, rmsnorm) or the sub-block's N(0, 4) beside a stream N(0, 1);
    weights are 1 + 0.1 N(0, 1) and 0.1 N(0, 1); incoming gradients N(0, 1)."""
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    rows, n, op = case["rows"], case["n"], case["op"]
    t = _TYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    def row_scaled():
        scale = 10.0 ** (4.0 * torch.rand(rows, 1, generator=g, device=dev) - 2.0)
        return ((normal(rows, n) + normal(rows, 1)) * scale).to(t)

    s = {"case": case, "rng": torch.randint(-2 ** 62, 2 ** 62, (2,), generator=g, device=dev,
                                            dtype=torch.int64),
         "site": 3, "gamma": (1.0 + 0.1 * normal(n)).to(t),
         "beta": (0.1 * normal(n)).to(t) if case["bias"] else None}
    if op == "layernorm":
        s["x"] = row_scaled()
    elif op in ("dropout_add", "dropout_add_layernorm"):
        s["x"] = (2.0 * normal(rows, n)).to(t)
        s["residual"] = normal(rows, n).to(t)
    else:
        s["dy"] = normal(rows, n).to(t)
        s["x"] = (normal(rows, n) + 0.5 * normal(rows, 1)).to(t) \
            if op == "dropout_add_layernorm_backward" else row_scaled()
        s["dstream"] = normal(rows, n).to(t) if case["dstream"] else None
    if op in ("layernorm_backward", "dropout_add_layernorm_backward"):
        s["mean"], s["rstd"] = _row_statistics(s["x"], case["eps"])

    # the buffers that a training loop keeps from step to step
    like = s["x"]
    if op == "layernorm":
        s["out"] = {"out": torch.empty_like(like)}
    elif op == "dropout_add":
        s["out"] = {"out": torch.empty_like(like)}
    elif op == "dropout_add_layernorm":
        s["out"] = {"out_stream": torch.empty_like(like), "normed": torch.empty_like(like)}
    else:
        s["out"] = {"dx": torch.empty_like(like), "dgamma": torch.empty(n, device=dev)}
        if op != "rmsnorm_backward":
            s["out"]["dbeta"] = torch.empty(n, device=dev) if case["bias"] else None
        if op == "dropout_add_layernorm_backward":
            s["out"]["dresidual"] = torch.empty_like(like)
        if own:
            from dual_epsilon_sandwich_gb300 import mrn
            s["workspace"] = mrn.norm_backward_workspace(s["x"])
    if op in ("layernorm", "dropout_add_layernorm"):
        s["out"]["mean"] = torch.empty(rows, device=dev)
        s["out"]["rstd"] = torch.empty(rows, device=dev)
    return s


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------
def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(s):
    from dual_epsilon_sandwich_gb300 import mrn
    c, o = s["case"], s["out"]
    op = c["op"]
    if op == "layernorm":
        mrn.layernorm(s["x"], s["gamma"], s["beta"], c["eps"], out=o["out"], mean=o["mean"],
                      rstd=o["rstd"])
    elif op == "dropout_add":
        mrn.dropout_add(s["x"], s["residual"], c["p"], s["rng"], site=s["site"], out=o["out"])
    elif op == "dropout_add_layernorm":
        mrn.dropout_add_layernorm(s["x"], s["residual"], s["gamma"], s["beta"], c["eps"], c["p"],
                                  s["rng"], site=s["site"], out_stream=o["out_stream"],
                                  normed=o["normed"], mean=o["mean"], rstd=o["rstd"])
    elif op == "layernorm_backward":
        mrn.layernorm_backward(s["dy"], s["x"], s["gamma"], s["mean"], s["rstd"],
                               dstream=s["dstream"], dx=o["dx"], dgamma=o["dgamma"],
                               dbeta=o["dbeta"], bias=c["bias"], workspace=s["workspace"])
    elif op == "dropout_add_layernorm_backward":
        mrn.dropout_add_layernorm_backward(
            s["dy"], s["x"], s["gamma"], s["mean"], s["rstd"], c["p"], s["rng"], site=s["site"],
            dstream=s["dstream"], dx=o["dx"], dresidual=o["dresidual"], dgamma=o["dgamma"],
            dbeta=o["dbeta"], bias=c["bias"], workspace=s["workspace"])
    else:
        mrn.rmsnorm_backward(s["dy"], s["x"], s["gamma"], c["eps"], dstream=s["dstream"],
                             dx=o["dx"], dgamma=o["dgamma"], workspace=s["workspace"])
    return {k: v for k, v in o.items() if v is not None}


def _row_statistics(x, eps):
    xf = x.float()
    n = x.shape[-1]
    mean = xf.sum(-1) / n
    d = xf - mean[:, None]
    return mean, 1.0 / torch.sqrt((d * d).sum(-1) / n + eps)


def _dropped(x, p, rng, site):
    """dropout(x) in f32 (plain form)."""
    t = int(p * 65536.0 + 0.5)
    if t == 0:
        return x.float()
    total = x.numel()
    low = 0xFFFFFFFF
    group = torch.arange((total + 7) // 8, device=x.device, dtype=torch.int64)
    step = rng[1] + site
    k0, k1 = rng[0] & low, (rng[0] >> 32) & low
    c0, c1 = group & low, group >> 32
    c2, c3 = (step & low).expand_as(group), ((step >> 32) & low).expand_as(group)
    for _ in range(10):
        # (the products wrap modulo 2^64; their upper words are bits 32..63 all the same)
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = (((b >> 32) & low) ^ c1 ^ k0, b & low,
                          ((a >> 32) & low) ^ c3 ^ k1, a & low)
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    lanes = []
    for word in (c0, c1, c2, c3):
        lanes += [word & 0xFFFF, word >> 16]
    u = torch.stack(lanes, dim=-1).reshape(-1)[:total].reshape(x.shape)
    scale = 65536.0 / (65536 - t) if t < 65536 else 0.0
    return torch.where(u >= t, x.float() * scale, torch.zeros((), device=x.device))


def _layernorm_plain(x, gamma, beta, eps):
    mean, rstd = _row_statistics(x, eps)
    y = (x.float() - mean[:, None]) * rstd[:, None] * gamma.float()
    if beta is not None:
        y = y + beta.float()
    return y, mean, rstd


def _layernorm_backward_plain(s):
    dy, x = s["dy"].float(), s["x"].float()
    n = x.shape[-1]
    rstd = s["rstd"][:, None]
    xh = (x - s["mean"][:, None]) * rstd
    w = dy * s["gamma"].float()
    dx = rstd * (w - w.sum(-1, keepdim=True) / n - xh * ((w * xh).sum(-1, keepdim=True) / n))
    if s["dstream"] is not None:
        dx = dx + s["dstream"].float()
    return dx, (dy * xh).sum(0), dy.sum(0)


def _run_plain(s):
    c = s["case"]
    op, t = c["op"], _TYPES[c["dtype"]]
    if op == "layernorm":
        y, mean, rstd = _layernorm_plain(s["x"], s["gamma"], s["beta"], c["eps"])
        return {"out": y.to(t), "mean": mean, "rstd": rstd}
    if op == "dropout_add":
        return {"out": (s["residual"].float() + _dropped(s["x"], c["p"], s["rng"],
                                                         s["site"])).to(t)}
    if op == "dropout_add_layernorm":
        stream = (s["residual"].float() + _dropped(s["x"], c["p"], s["rng"], s["site"])).to(t)
        y, mean, rstd = _layernorm_plain(stream, s["gamma"], s["beta"], c["eps"])
        return {"out_stream": stream, "normed": y.to(t), "mean": mean, "rstd": rstd}
    if op == "rmsnorm_backward":
        dy, x = s["dy"].float(), s["x"].float()
        n = x.shape[-1]
        inv = 1.0 / torch.sqrt((x * x).sum(-1, keepdim=True) / n + c["eps"])
        w = dy * s["gamma"].float()
        xh = x * inv
        dx = inv * (w - xh * ((w * xh).sum(-1, keepdim=True) / n))
        if s["dstream"] is not None:
            dx = dx + s["dstream"].float()
        return {"dx": dx.to(t), "dgamma": (dy * xh).sum(0)}
    dx, dgamma, dbeta = _layernorm_backward_plain(s)
    out = {"dx": dx.to(t), "dgamma": dgamma}
    if c["bias"]:
        out["dbeta"] = dbeta
    if op == "dropout_add_layernorm_backward":
        out["dx"] = _dropped(dx, c["p"], s["rng"], s["site"]).to(t)
        out["dresidual"] = dx.to(t)
    return out


# ---------------------------------------------------------------------------
# The definition in 64 bits
# ---------------------------------------------------------------------------
def _mulhilo(a, m):
    """(upper, lower) word of the 32 x 32 bit product, from 16-bit limbs."""
    al, ah, ml, mh = a & 0xFFFF, a >> 16, m & 0xFFFF, m >> 16
    ll, lh, hl, hh = al * ml, al * mh, ah * ml, ah * mh
    mid = (ll >> 16) + (lh & 0xFFFF) + (hl & 0xFFFF)
    return hh + (lh >> 16) + (hl >> 16) + (mid >> 16), ((mid & 0xFFFF) << 16) | (ll & 0xFFFF)


def _kept(shape, p, rng, site, device):
    """Truth values: the elements that a dropout keeps."""
    total = math.prod(shape)
    seed, step = (int(v) & (2 ** 64 - 1) for v in rng.tolist())
    step = (step + site) & (2 ** 64 - 1)
    e = torch.arange(0, total + 7, 8, device=device, dtype=torch.int64)[:(total + 7) // 8] // 8
    ctr = [e % 2 ** 32, e // 2 ** 32, torch.full_like(e, step % 2 ** 32),
           torch.full_like(e, step // 2 ** 32)]
    for i in range(10):
        key = ((seed % 2 ** 32 + i * 0x9E3779B9) % 2 ** 32,
               (seed // 2 ** 32 + i * 0xBB67AE85) % 2 ** 32)
        h0, l0 = _mulhilo(ctr[0], 0xD2511F53)
        h1, l1 = _mulhilo(ctr[2], 0xCD9E8D57)
        ctr = [h1 ^ ctr[1] ^ key[0], l1, h0 ^ ctr[3] ^ key[1], l0]
    t = math.floor(p * 65536 + 0.5)
    keep = torch.empty(len(e), 8, dtype=torch.bool, device=device)
    for lane in range(8):
        keep[:, lane] = (ctr[lane // 2] // 2 ** (16 * (lane % 2))) % 2 ** 16 >= t
    return keep.view(-1)[:total].view(shape), (65536 / (65536 - t) if t < 65536 else 0.0)


def exact(case, seed):
    s = prepare(case, seed)
    op, n, t = case["op"], case["n"], _TYPES[case["dtype"]]
    x, gamma = s["x"].double(), s["gamma"].double()
    beta = s["beta"].double() if s["beta"] is not None else torch.zeros_like(gamma)

    def norm(v):
        mean = v.mean(-1, keepdim=True)
        rstd = ((v - mean).square().mean(-1, keepdim=True) + case["eps"]).rsqrt()
        return (v - mean) * rstd * gamma + beta, mean[:, 0], rstd[:, 0]

    if op == "layernorm":
        y, mean, rstd = norm(x)
        return {"out": y, "mean": mean, "rstd": rstd}
    if op in ("dropout_add", "dropout_add_layernorm"):
        keep, scale = _kept(x.shape, case["p"], s["rng"], s["site"], x.device)
        stream = s["residual"].double() + torch.where(keep, x * scale, 0.0)
        if op == "dropout_add":
            return {"out": stream}
        y, mean, rstd = norm(stream.to(t).double())
        return {"out_stream": stream, "normed": y, "mean": mean, "rstd": rstd}
    dy = s["dy"].double()
    if op == "rmsnorm_backward":
        mean = torch.zeros_like(x[:, :1])
        rstd = (x.square().mean(-1, keepdim=True) + case["eps"]).rsqrt()
    else:
        mean, rstd = s["mean"].double()[:, None], s["rstd"].double()[:, None]
    xh = (x - mean) * rstd
    w = dy * gamma
    dx = w - xh * (w * xh).mean(-1, keepdim=True)
    if op != "rmsnorm_backward":
        dx -= w.mean(-1, keepdim=True)
    dx *= rstd
    if s["dstream"] is not None:
        dx += s["dstream"].double()
    out = {"dx": dx, "dgamma": (dy * xh).sum(0)}
    if op != "rmsnorm_backward" and case["bias"]:
        out["dbeta"] = dy.sum(0)
    if op == "dropout_add_layernorm_backward":
        keep, scale = _kept(x.shape, case["p"], s["rng"], s["site"], x.device)
        out["dx"] = torch.where(keep, dx * scale, 0.0)
        out["dresidual"] = dx
    return out


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    rows, n, op = case["rows"], case["n"], case["op"]
    size = 4 if case["dtype"] == "f32" else 2
    matrices = {"layernorm": 2, "dropout_add": 3, "dropout_add_layernorm": 4,
                "layernorm_backward": 3, "dropout_add_layernorm_backward": 4,
                "rmsnorm_backward": 3}[op]
    per_element = {"layernorm": 7, "dropout_add": 2, "dropout_add_layernorm": 9,
                   "layernorm_backward": 14, "dropout_add_layernorm_backward": 15,
                   "rmsnorm_backward": 11}[op]
    if op.endswith("backward") and case["dstream"]:
        matrices += 1
        per_element += 1
    total = matrices * rows * n * size
    if op != "dropout_add":
        total += n * size                                  # gamma
    if op in ("layernorm", "dropout_add_layernorm"):
        total += 8 * rows + (n * size if case["bias"] else 0)
    elif op in ("layernorm_backward", "dropout_add_layernorm_backward"):
        total += 8 * rows + 4 * n + (4 * n if case["bias"] else 0)
    elif op == "rmsnorm_backward":
        total += 4 * n
    return {"bytes": total, "flops": per_element * rows * n}
