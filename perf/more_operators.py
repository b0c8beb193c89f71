"""Cases of what trains the dense student of the exact lists in less memory: the
cross entropy over every item without its logits, and activations kept in 8
bits for the gradients.

Each case is one pass of one operator.  ``run`` computes it in plain torch
operations in 32 bits, or, with ``own`` true, through the library's calls.

  xent      loss_r = weight_r (log sum_v exp(z_rv) - z_r[target_r]) with
            z = (x w^T + bias) / T over every item, and with it its gradients
            for x, w and bias; a row without a target, with one that the bias
            masks (-inf), or of weight 0 has loss 0 and gradient 0
  compress  values to e4m3 with a power of two for every 32 of a row (the
            smallest that brings them to 448 or less), and back
  keep      a linear layer y = act(x w^T + bias) whose pre-activation is kept
            so for the gradient
  layer     that layer's gradients from its input and pre-activation kept so
  norm      the root-mean-square norm's gradient from its summed input kept so
"""
import functools
import math

import torch

own = False

F8_MAX = 448.0
GROUP = 32
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
# the smallest exponents of a group's scale, for which code times scale is a value of the type
LEAST = {"bf16": -124, "f16": -15, "f32": -126}
ACTIVATIONS = ("none", "relu", "gelu", "gelu_tanh", "silu", "log1p_relu")
MOST_STEP = 2500 * 200_000 * 1024
MOST_LOSS = 5000 * 200_000 * 1024
MOST_LAYER = 8192 * 4096 * 1024
EPS = 1e-6


def listed():
    return [
        # A few queries' losses over the 10,000 items of the small workload, as
        # a training run watches them: latency counts.
        dict(name="xent_queries", op="xent", m=16, v=10_000, k=256, type="bf16", masked=False, temperature=1.0,
             grad=False, fused=False),
        # The losses of the 5,000 queries over the 200,000 items of the
        # throughput workload.
        dict(name="xent_eval", op="xent", m=5000, v=200_000, k=1024, type="bf16", masked=False, temperature=1.0,
             grad=False, fused=False),
        # A training step of 512 queries over 10,000 items at width 256, the
        # sizes of the student's example.
        dict(name="xent_student", op="xent", m=512, v=10_000, k=256, type="bf16", masked=True, temperature=1.0,
             grad=True, fused=True),
        # Odd everything: rows that start on no 16-byte boundary, a temperature
        # as normalised vectors have one, loss and gradient in two calls.
        dict(name="xent_ragged", op="xent", m=1003, v=50_001, k=777, type="f16", masked=True, temperature=0.5,
             grad=True, fused=False),
        # A training step of half of the 5,000 queries over the 200,000 items.
        dict(name="xent_step", op="xent", m=2500, v=200_000, k=1024, type="bf16", masked=False, temperature=1.0,
             grad=True, fused=True),
        # Four rows' values kept and given back: two short launches.
        dict(name="compress_rows", op="compress", rows=4, cols=4096, type="bf16"),
        # A long batch's activations kept and given back.
        dict(name="compress_batch", op="compress", rows=16_384, cols=4096, type="bf16"),
        # A training batch's projection that keeps its pre-activation in 8 bits.
        dict(name="keep_batch", op="keep", m=8192, k=1024, n=4096, type="bf16", act="gelu"),
        # Odd everything, kept in rows that start anywhere.
        dict(name="layer_ragged", op="layer", m=1003, k=1001, n=777, type="f16", act="silu"),
        # The gradients of a training batch's projection from what it kept.
        dict(name="layer_batch", op="layer", m=8192, k=1024, n=4096, type="bf16", act="gelu"),
        # The norm's gradient for a batch of an odd width.
        dict(name="norm_odd", op="norm", rows=5000, cols=1001, type="f32", residual=True),
        # The norm's gradient for a training batch.
        dict(name="norm_batch", op="norm", rows=16_384, cols=2048, type="bf16", residual=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["xent", "xent", "xent", "compress", "keep", "layer", "norm"])
    whole = rng.random() < 0.5  # widths of whole 16-byte units, or any other
    if op == "xent":
        grad = rng.random() < 0.6
        k, v = _log(rng, 64, 2048), _log(rng, 500, 200_000)
        if whole:
            k, v = k // 8 * 8, v // 8 * 8
        most = MOST_STEP if grad else MOST_LOSS
        m = max(1, min(_log(rng, 1, 5000), most // (v * k), most // 1024 // v))
        return dict(op="xent", m=m, v=v, k=k, type=rng.choice(["bf16", "f16"]), masked=rng.random() < 0.5,
                    temperature=rng.choice([0.5, 1.0, 2.0]), grad=grad, fused=grad and rng.random() < 0.6)
    if op in ("keep", "layer"):
        k, n = _log(rng, 128, 4096), _log(rng, 128, 10_000)
        if whole:
            k, n = k // 16 * 16, n // 16 * 16
        m = max(1, min(_log(rng, 1, 8192), MOST_LAYER // (n * k)))
        return dict(op=op, m=m, k=k, n=n, type=rng.choice(["bf16", "f16"]), act=rng.choice(ACTIVATIONS[1:]))
    cols = _log(rng, 128, 16_384 if op == "norm" else 65_536)
    if whole:
        cols = cols // 32 * 32
    rows = max(1, min(_log(rng, 1, 16_384), 16_384 * (2048 if op == "norm" else 4096) // cols))
    case = dict(op=op, rows=rows, cols=cols, type=rng.choice(["bf16", "f16", "f32"]))
    return dict(case, residual=rng.random() < 0.7) if op == "norm" else case


def _normal(g, shape, std=1.0, dtype=torch.float32):
    x = torch.empty(shape, dtype=dtype, device="cuda")
    return x.normal_(0.0, std, generator=g)


def _power(e):
    """2^e in float32, -126 <= e <= 127, from the exponent's bits."""
    return ((e + 127) << 23).view(torch.float32)


def _codes(x, least):
    """(codes in float32, exponents of the groups) of a float32 matrix."""
    rows, cols = x.shape
    groups = (cols + GROUP - 1) // GROUP
    full = torch.zeros((rows, groups * GROUP), device=x.device)
    full[:, :cols] = x
    full = full.view(rows, groups, GROUP)
    finite = torch.where(torch.isfinite(full), full.abs(), torch.zeros_like(full))
    mantissa, exponent = torch.frexp(finite.amax(2))  # in [1/2, 1)
    e = (exponent - 9 + (mantissa > 0.875)).clamp_min(least)
    q = torch.where(torch.isfinite(full), full, torch.full_like(full, math.nan)) * _power(-e)[:, :, None]
    return q.to(torch.float8_e4m3fn).view(rows, -1)[:, :cols].contiguous(), e


def _values(codes, e):
    """What codes and exponents stand for, in float32."""
    cols = codes.shape[1]
    return codes.float() * _power(e).repeat_interleave(GROUP, dim=1)[:, :cols]


def _kept(x, name):
    """A matrix as the forward pass keeps it: codes, scales and exponents."""
    codes, e = _codes(x.float(), LEAST[name])
    return codes, (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu), e


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    st = dict(case=case)
    op, t = case["op"], TYPES[case["type"]]
    if op == "xent":
        m, v, k = case["m"], case["v"], case["k"]
        st["x"], st["w"] = _normal(g, (m, k), 1.0, t), _normal(g, (v, k), 2.5 * case["temperature"] * k ** -0.5, t)
        st["bias"] = _normal(g, (v,), 0.3)
        if case["masked"]:  # items that the student may not answer
            st["bias"][torch.randint(0, v, (max(1, v // 100),), generator=g, device="cuda")] = -math.inf
        st["targets"] = torch.randint(0, v, (m,), generator=g, device="cuda")
        padding = torch.rand((m,), generator=g, device="cuda")
        if m > 1:
            st["targets"] = st["targets"].masked_fill(padding < 0.03, -1)
        st["weight"] = (torch.rand((m,), generator=g, device="cuda") + 0.5).masked_fill(padding > 0.98, 0.0)
        # the mean's gradient, with a loss scale where the gradients have 5 bits of exponent
        st["grad_loss"] = torch.full((m,), (1024.0 if case["type"] == "f16" else 1.0) / m, device="cuda")
    elif op == "compress":
        x = _normal(g, (case["rows"], case["cols"]))
        # activations: a few features much larger than the others
        st["x"] = (x * (1 + 30 * (torch.rand((case["cols"],), generator=g, device="cuda") < 0.01))).to(t)
    elif op in ("keep", "layer"):
        m, k, n = case["m"], case["k"], case["n"]
        x = _normal(g, (m, k), 1.0, t)
        st["w"], st["bias"] = _normal(g, (n, k), k ** -0.5, t), _normal(g, (n,), 0.1)
        if op == "keep":
            st["x"] = x
        else:
            st["x"], st["x_scale"], st["x_exponent"] = _kept(x, case["type"])
            pre = x.float() @ st["w"].float().t() + st["bias"]
            st["pre"], st["pre_scale"], st["pre_exponent"] = _kept(pre, case["type"])
            st["grad_y"] = _normal(g, (m, n), 1.0 if case["type"] == "f16" else 1.0 / n, t)
    else:
        r, c = case["rows"], case["cols"]
        total = _normal(g, (r, c), 2.0, t)
        st["rstd"] = torch.rsqrt(total.float().square().mean(1) + EPS)
        st["total"], st["total_scale"], st["total_exponent"] = _kept(total, case["type"])
        st["weight"] = 1.0 + _normal(g, (c,), 0.1)
        st["grad_y"] = _normal(g, (r, c), 0.5, t)
        st["grad_total"] = _normal(g, (r, c), 0.5, t) if case["residual"] else None
    return st


# ---------------------------------------------------------------- plain forms
def _act(z, name):
    if name == "relu":
        return torch.clamp_min(z, 0)
    if name == "gelu":
        return 0.5 * z * (1 + torch.erf(z * 0.5 ** 0.5))
    if name == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh((2 / math.pi) ** 0.5 * (z + 0.044715 * z ** 3)))
    if name == "silu":
        return z / (1 + torch.exp(-z))
    return torch.log1p(torch.clamp_min(z, 0))


def _slope(z, name):
    if name == "relu":
        return (z > 0).float()
    if name == "gelu":
        return 0.5 * (1 + torch.erf(z * 0.5 ** 0.5)) + z * torch.exp(-0.5 * z * z) / (2 * math.pi) ** 0.5
    if name == "gelu_tanh":
        c = (2 / math.pi) ** 0.5
        t = torch.tanh(c * (z + 0.044715 * z ** 3))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)
    if name == "silu":
        s = 1 / (1 + torch.exp(-z))
        return s * (1 + z * (1 - s))
    return torch.where(z > 0, 1 / (1 + torch.clamp_min(z, 0)), torch.zeros_like(z))


def _plain_xent(st):
    c, T, t = st["case"], st["case"]["temperature"], st["x"].dtype
    x, w = st["x"].float(), st["w"].float()
    z = (x @ w.t() + st["bias"]) / T
    at = st["targets"].clamp_min(0)[:, None]
    here = torch.gather(z, 1, at)
    live = (st["targets"] >= 0) & (here[:, 0] > -math.inf) & (st["weight"] != 0)
    most = z.amax(1, keepdim=True)
    e = torch.exp(z - most)
    total = e.sum(1, keepdim=True)
    loss = st["weight"] * (torch.log(total) - (here - most))[:, 0]
    loss = torch.where(live, loss, torch.zeros_like(loss))
    if not c["grad"]:
        return {"loss": loss}
    scale = torch.where(live, st["weight"] * st["grad_loss"] / T, torch.zeros_like(loss))
    gz = (e / total).scatter_add(1, at, torch.full_like(here, -1.0))
    gz = torch.where(live[:, None], gz * scale[:, None], torch.zeros_like(gz))
    return {"loss": loss, "grad_x": (gz @ w).to(t), "grad_w": (gz.t() @ x).to(t), "grad_bias": gz.sum(0)}


def _plain_compress(st):
    codes, e = _codes(st["x"].float(), LEAST[st["case"]["type"]])
    return {"values": _values(codes, e).to(st["x"].dtype)}


def _plain_keep(st):
    c, t = st["case"], st["x"].dtype
    z = st["x"].float() @ st["w"].float().t() + st["bias"]
    codes, e = _codes(z, LEAST[c["type"]])
    return {"y": _act(z, c["act"]).to(t), "pre": _values(codes, e).to(t)}


def _plain_layer(st):
    c, t = st["case"], st["w"].dtype
    x, w = _values(st["x"], st["x_exponent"]), st["w"].float()
    gz = st["grad_y"].float() * _slope(_values(st["pre"], st["pre_exponent"]), c["act"])
    return {"grad_x": (gz @ w).to(t), "grad_w": (gz.t() @ x).to(t), "grad_bias": gz.sum(0)}


def _plain_norm(st):
    t = st["grad_y"].dtype
    gy, xhat = st["grad_y"].float(), _values(st["total"], st["total_exponent"]) * st["rstd"][:, None]
    g = gy * st["weight"]
    gx = st["rstd"][:, None] * (g - xhat * (g * xhat).mean(1, keepdim=True))
    if st["grad_total"] is not None:
        gx = gx + st["grad_total"].float()
    return {"grad_x": gx.to(t), "grad_weight": (gy * xhat).sum(0)}


# ---------------------------------------------------------------- the library
@functools.lru_cache(maxsize=1)
def _handle():
    import sparse_embedding_exact_gb300 as sec

    return sec.SparseCosine(65_536, chunk_rows=256)


def _own(st):
    h, c = _handle(), st["case"]
    if c["op"] == "xent":
        more = dict(bias=st["bias"], weight=st["weight"], temperature=c["temperature"])
        if c["fused"]:
            loss, gx, gw, gb = h.cross_entropy_step(st["x"], st["w"], st["targets"], st["grad_loss"], **more)
        else:
            loss, stats = h.cross_entropy(st["x"], st["w"], st["targets"], **more)
            if not c["grad"]:
                return {"loss": loss}
            gx, gw, gb = h.cross_entropy_backward(st["grad_loss"], st["x"], st["w"], st["targets"], stats, **more)
        return {"loss": loss, "grad_x": gx, "grad_w": gw, "grad_bias": gb}
    if c["op"] == "compress":
        codes, scale = h.compress(st["x"])
        return {"values": h.expand(codes, scale, st["x"].dtype)}
    if c["op"] == "keep":
        y, pre, scale = h.linear(st["x"], st["w"], bias=st["bias"], activation=c["act"], compress_pre=True)
        return {"y": y, "pre": h.expand(pre, scale, st["x"].dtype)}
    if c["op"] == "layer":
        gx, gw, gb = h.linear_backward(st["grad_y"], st["x"], st["w"], pre=st["pre"], activation=c["act"],
                                       x_scale=st["x_scale"], pre_scale=st["pre_scale"])
        return {"grad_x": gx, "grad_w": gw, "grad_bias": gb}
    gx, gw = h.rms_norm_backward(st["grad_y"], st["total"], st["weight"], st["rstd"], grad_total=st["grad_total"],
                                 total_scale=st["total_scale"])
    return {"grad_x": gx, "grad_weight": gw}


def run(state):
    if own:
        return _own(state)
    return {"xent": _plain_xent, "compress": _plain_compress, "keep": _plain_keep, "layer": _plain_layer,
            "norm": _plain_norm}[state["case"]["op"]](state)


def work(case):
    op, size = case["op"], 4 if case["type"] == "f32" else 2
    if op == "xent":
        m, v, k = case["m"], case["v"], case["k"]
        b = (m * k + v * k) * size + 4 * v + m * (8 + 4 + 4)
        if case["grad"]:
            b += (m * k + v * k) * size + 4 * v + 4 * m
        return {"bytes": b, "flops": (6 if case["grad"] else 2) * m * v * k}
    if op in ("keep", "layer"):
        m, k, n = case["m"], case["k"], case["n"]
        kept = lambda r, c: r * c + r * ((c + GROUP - 1) // GROUP)  # noqa: E731
        if op == "keep":  # the kept values once more, read and given back
            return {"bytes": (m * k + n * k) * size + 4 * n + 2 * m * n * size + 2 * kept(m, n), "flops": 2 * m * n * k}
        b = kept(m, k) + kept(m, n) + (n * k + m * n) * size + (m * k + n * k) * size + 4 * n
        return {"bytes": b, "flops": 4 * m * n * k}
    e, groups = case["rows"] * case["cols"], case["rows"] * ((case["cols"] + GROUP - 1) // GROUP)
    if op == "compress":
        return {"bytes": 2 * (e * size + e + groups), "flops": 3 * e}
    return {"bytes": e * size * (3 if case["residual"] else 2) + e + groups + 8 * case["cols"] + 4 * case["rows"],
            "flops": 10 * e}


# ------------------------------------------------ the definitions in 64 bits
def _nearest_code(q):
    """The nearest value of 3 bits after the point, 2^-9 the smallest."""
    unit = torch.exp2(torch.floor(torch.log2(q.abs().clamp_min(2.0 ** -6))) - 3)
    return torch.round(q / unit) * unit


def _compressed_exactly(x, least):
    """What a matrix of 64 bits stands for once it has been compressed."""
    cols = x.shape[1]
    parts = torch.nn.functional.pad(x, (0, -cols % GROUP)).unflatten(1, (-1, GROUP))
    most = torch.linalg.vector_norm(parts, ord=math.inf, dim=2, keepdim=True)
    e = torch.ceil(torch.log2(most / F8_MAX)).clamp_min(least)
    return (_nearest_code(parts * torch.exp2(-e)) * torch.exp2(e)).flatten(1)[:, :cols]


def _stands_for(codes, scale):
    s = torch.exp2(scale.view(torch.uint8).double() - 127)
    column = torch.arange(codes.shape[1], device=codes.device) // GROUP
    return codes.double() * s[:, column]


def exact(case, seed):
    st = prepare(case, seed)
    d, op = torch.float64, case["op"]
    if op == "xent":
        T = case["temperature"]
        if 6.0 * case["m"] * case["v"] * case["k"] > 7e12:
            return None
        x, w = st["x"].to(d), st["w"].to(d)
        log_q = torch.log_softmax(torch.addmm(st["bias"].to(d), x, w.t()) / T, 1)
        rows = torch.arange(case["m"], device="cuda")
        best = st["targets"].clamp_min(0)
        at, weight = log_q[rows, best], st["weight"].to(d)
        ok = (st["targets"] >= 0) & torch.isfinite(at) & (weight != 0)
        loss = torch.where(ok, -weight * at, torch.zeros_like(at))
        if not case["grad"]:
            return {"loss": loss}
        gz = log_q.exp_()
        gz[rows, best] -= 1
        gz *= torch.where(ok, weight * st["grad_loss"].to(d) / T, torch.zeros_like(at))[:, None]
        return {"loss": loss, "grad_x": torch.mm(gz, w), "grad_w": torch.mm(gz.t(), x), "grad_bias": gz.sum(0)}
    if op == "compress":
        return {"values": _compressed_exactly(st["x"].to(d), LEAST[case["type"]])}
    if op in ("keep", "layer"):
        name = case["act"]
        act = {"relu": torch.relu, "gelu": torch.nn.functional.gelu,
               "gelu_tanh": lambda z: torch.nn.functional.gelu(z, approximate="tanh"),
               "silu": torch.nn.functional.silu, "log1p_relu": lambda z: torch.relu(z).log1p()}[name]
        w = st["w"].to(d)
        if op == "keep":
            z = torch.addmm(st["bias"].to(d), st["x"].to(d), w.t())
            return {"y": act(z), "pre": _compressed_exactly(z, LEAST[case["type"]])}
        x, z = _stands_for(st["x"], st["x_scale"]), _stands_for(st["pre"], st["pre_scale"]).requires_grad_()
        gz, = torch.autograd.grad(act(z), z, st["grad_y"].to(d))
        return {"grad_x": torch.mm(gz, w), "grad_w": torch.mm(gz.t(), x), "grad_bias": gz.sum(0)}
    s, w, gy = _stands_for(st["total"], st["total_scale"]), st["weight"].to(d), st["grad_y"].to(d)
    rstd = st["rstd"].to(d)[:, None]
    dot = torch.einsum("rc,rc,c->r", gy, s, w)[:, None]
    gx = rstd * gy * w - s * rstd ** 3 * dot / case["cols"]
    if st["grad_total"] is not None:
        gx += st["grad_total"].to(d)
    return {"grad_x": gx, "grad_weight": torch.einsum("rc,rc,r->c", gy, s, rstd[:, 0])}
