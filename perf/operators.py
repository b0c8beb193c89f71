"""Cases of the dense student operators: normalisation, linear layers and the
distillation loss that train and serve a dense student of the exact top-k lists.

Each case is one pass of one operator.  ``run`` computes it in plain torch
operations in 32 bits, or, with ``own`` true, through the library's calls.

  rms_norm   s = x + r;  y = s / sqrt(mean(s^2) + eps) * w, also with an output
             in 8 bits (e4m3) and one scale a row; and its gradient
  linear     y = act((x w^T) sx sw^T + b) + r, inputs in 16 bits or in 8 bits
             with one scale a row; and its gradient
  distill    loss_r = weight_r T^2 KL(p_r || q_r), p_r the softmax of a
             teacher's k listed scores over U, q_r the softmax of the student's
             logits over T over every item; and its gradient
"""
import functools
import math

import torch

own = False

F8_MAX = 448.0
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
ACTIVATIONS = ("none", "relu", "gelu", "gelu_tanh", "silu", "log1p_relu")
MOST_FLOPS = 2.0 * 8192 * 4096 * 4096
MOST_LOGITS = 2500 * 200_000
EPS = 1e-6


def listed():
    return [
        # One query's sparse embedding over the 65,536 dimensions of the small
        # workload: log(1 + relu) of a vocabulary head, weights read once.
        dict(name="linear_token_head", op="linear", m=1, k=1024, n=65_536, type="bf16", act="log1p_relu",
             residual=False, grad=False),
        # A serving batch of 16 tokens through an 8-bit layer: latency counts.
        dict(name="linear_f8_tokens", op="linear", m=16, k=4096, n=4096, type="f8", act="none",
             residual=True, grad=False),
        # Odd everything: rows that start on no 16-byte boundary.
        dict(name="linear_ragged", op="linear", m=1003, k=1001, n=777, type="f16", act="silu",
             residual=True, grad=False),
        # A training batch's projection, the pre-activation kept for the gradient.
        dict(name="linear_train", op="linear", m=8192, k=4096, n=4096, type="bf16", act="gelu",
             residual=True, grad=False),
        # The gradients of a training batch's projection.
        dict(name="linear_train_grad", op="linear", m=8192, k=1024, n=4096, type="bf16", act="gelu",
             residual=False, grad=True),
        # 8-bit scoring of 5,000 queries against 10,000 items' dense vectors.
        dict(name="linear_f8_logits", op="linear", m=5000, k=2048, n=10_000, type="f8", act="none",
             residual=False, grad=False),
        # The norm before an 8-bit layer for four tokens: one short launch.
        dict(name="rms_f8_tokens", op="rms", rows=4, cols=4096, type="bf16", residual=True, out="f8", grad=False),
        # The same over a long batch.
        dict(name="rms_f8_batch", op="rms", rows=16_384, cols=4096, type="bf16", residual=True, out="f8", grad=False),
        # Its gradient for a training batch of an odd width (no row but the
        # first on a 16-byte boundary).
        dict(name="rms_grad_odd", op="rms", rows=5000, cols=1001, type="f32", residual=True, out="same", grad=True),
        # Its gradient for a training batch.
        dict(name="rms_grad", op="rms", rows=16_384, cols=2048, type="bf16", residual=True, out="same", grad=True),
        # One small batch over the 10,000 items of the small workload, top 10.
        dict(name="distill_small", op="distill", rows=64, items=10_000, k=10, type="f32", masked=True,
             temperature=1.0, fused=True),
        # Half of the 5,000 queries x 200,000 items of the throughput workload,
        # top 64: loss and gradient of a training step.
        dict(name="distill_step", op="distill", rows=2500, items=200_000, k=64, type="bf16", masked=False,
             temperature=1.0, fused=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["linear", "linear", "rms", "distill"])
    if op == "linear":
        kind = rng.choice(["token", "batch", "grad"])
        t = rng.choice(["bf16", "f16"] if kind == "grad" else ["bf16", "f16", "f8"])
        k, n = _log(rng, 256, 4096), _log(rng, 256, 65_536 if kind == "token" else 10_000)
        if t == "f8" or rng.random() < 0.5:  # widths of whole 16-byte units, and any other
            k, n = k // 16 * 16 | 16, n // 16 * 16 | 16
        m = _log(rng, 1, 64) if kind == "token" else _log(rng, 65, 8192)
        m = max(1, min(m, int(MOST_FLOPS / (2.0 * n * k * (2 if kind == "grad" else 1)))))
        act = rng.choice(ACTIVATIONS)
        return dict(op="linear", m=m, k=k, n=n, type=t, act=act, residual=kind != "grad" and rng.random() < 0.5,
                    grad=kind == "grad")
    if op == "rms":
        cols = _log(rng, 128, 16_384)
        if rng.random() < 0.5:
            cols = cols // 8 * 8 | 8
        rows = max(1, min(_log(rng, 1, 16_384), 16_384 * 4096 // cols))
        grad = rng.random() < 0.4
        return dict(op="rms", rows=rows, cols=cols, type=rng.choice(["bf16", "f16", "f32"]),
                    residual=rng.random() < 0.7, out="same" if grad else rng.choice(["same", "f8"]), grad=grad)
    items = _log(rng, 500, 500_000)
    rows = max(1, min(_log(rng, 1, 5000), MOST_LOGITS // items))
    return dict(op="distill", rows=rows, items=items, k=_log(rng, 1, 64), type=rng.choice(["bf16", "f16", "f32"]),
                masked=rng.random() < 0.5, temperature=rng.choice([0.5, 1.0, 2.0]), fused=rng.random() < 0.6)


def _normal(g, shape, std=1.0, dtype=torch.float32):
    x = torch.empty(shape, dtype=dtype, device="cuda")
    return x.normal_(0.0, std, generator=g)


def _quantized(x):
    """A matrix in e4m3 with one scale a row, as it is kept or handed on."""
    scale = x.abs().amax(1) / F8_MAX
    return (x / scale[:, None]).clamp(-F8_MAX, F8_MAX).to(torch.float8_e4m3fn), scale


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    st = dict(case=case)
    if case["op"] == "linear":
        m, k, n = case["m"], case["k"], case["n"]
        t = TYPES.get(case["type"], torch.bfloat16)
        if case["type"] == "f8":
            st["x"], st["x_scale"] = _quantized(_normal(g, (m, k)))
            st["w"], st["w_scale"] = _quantized(_normal(g, (n, k), k ** -0.5))
        else:
            st["x"], st["w"] = _normal(g, (m, k), 1.0, t), _normal(g, (n, k), k ** -0.5, t)
        st["bias"] = _normal(g, (n,), 0.1)
        st["residual"] = _normal(g, (m, n), 1.0, t) if case["residual"] else None
        if case["grad"]:
            st["grad_y"] = _normal(g, (m, n), 1.0 / n, t) if t != torch.float16 else _normal(g, (m, n), 1.0, t)
            # the pre-activation that the forward pass of these inputs keeps
            st["pre"] = (st["x"].float() @ st["w"].float().t() + st["bias"]).to(t)
    elif case["op"] == "rms":
        r, c, t = case["rows"], case["cols"], TYPES[case["type"]]
        st["weight"] = 1.0 + _normal(g, (c,), 0.1)
        if t != torch.float32:
            st["weight"] = st["weight"].to(t)
        if case["grad"]:
            st["total"] = _normal(g, (r, c), 2.0, t)
            st["rstd"] = torch.rsqrt(st["total"].float().square().mean(1) + EPS)
            st["grad_y"] = _normal(g, (r, c), 0.5, t)
            st["grad_total"] = _normal(g, (r, c), 0.5, t) if case["residual"] else None
        else:
            st["x"] = _normal(g, (r, c), 1.0, t)
            st["residual"] = _normal(g, (r, c), 2.0, t) if case["residual"] else None
    else:
        r, v, k = case["rows"], case["items"], case["k"]
        st["logits"] = _normal(g, (r, v), 2.5, TYPES[case["type"]])
        step = 7919 if v % 7919 else 7907
        first = torch.randint(0, v, (r, 1), generator=g, device="cuda")
        st["best"] = (first + torch.arange(k, device="cuda") * step) % v  # distinct items
        s = torch.rand((r, k), generator=g, device="cuda")
        st["scores"] = s.sort(1, descending=True).values  # cosines, the best first
        have = torch.randint(0, 4 * k, (r, 1), generator=g, device="cuda")
        absent = torch.arange(k, device="cuda") > have  # lists that end early
        st["best"] = st["best"].masked_fill(absent, -1)
        st["scores"] = st["scores"].masked_fill(absent, -math.inf)
        st["weight"] = (torch.rand((r,), generator=g, device="cuda") < 0.95).float()  # padding rows: 0
        # the mean's gradient, with a loss scale where the gradient has 5 bits of exponent
        st["grad_loss"] = torch.full((r,), (1024.0 if case["type"] == "f16" else 1.0) / r, device="cuda")
        if case["masked"]:  # items that the student may not answer
            at = torch.randint(0, v, (max(1, v // 100),), generator=g, device="cuda")
            st["logits"][:, at] = -math.inf
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
        return z * torch.sigmoid(z)
    if name == "log1p_relu":
        return torch.log1p(torch.clamp_min(z, 0))
    return z


def _act_slope(z, name):
    if name == "relu":
        return (z > 0).float()
    if name == "gelu":
        return 0.5 * (1 + torch.erf(z * 0.5 ** 0.5)) + z * torch.exp(-0.5 * z * z) / (2 * math.pi) ** 0.5
    if name == "gelu_tanh":
        c = (2 / math.pi) ** 0.5
        t = torch.tanh(c * (z + 0.044715 * z ** 3))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)
    if name == "silu":
        s = torch.sigmoid(z)
        return s * (1 + z * (1 - s))
    if name == "log1p_relu":
        return torch.where(z > 0, 1 / (1 + torch.clamp_min(z, 0)), torch.zeros_like(z))
    return torch.ones_like(z)


def _plain_linear(st):
    c = st["case"]
    x, w = st["x"].float(), st["w"].float()
    if c["grad"]:
        t = st["x"].dtype
        gz = st["grad_y"].float()
        if c["act"] != "none":
            gz = gz * _act_slope(st["pre"].float(), c["act"])
        return {"grad_x": (gz @ w).to(t), "grad_w": (gz.t() @ x).to(t), "grad_bias": gz.sum(0)}
    z = x @ w.t()
    t = st["x"].dtype
    if c["type"] == "f8":
        z = z * st["x_scale"][:, None] * st["w_scale"]
        t = torch.bfloat16
    z = z + st["bias"]
    y = _act(z, c["act"])
    if st["residual"] is not None:
        y = y + st["residual"].float()
    if c["act"] in ("gelu", "gelu_tanh", "silu"):  # kept for the gradient
        return {"y": y.to(t), "pre": z.to(t)}
    return {"y": y.to(t)}


def _plain_rms(st):
    c = st["case"]
    w = st["weight"].float()
    if c["grad"]:
        t = st["total"].dtype
        gy, xhat = st["grad_y"].float(), st["total"].float() * st["rstd"][:, None]
        g = gy * w
        gx = st["rstd"][:, None] * (g - xhat * (g * xhat).mean(1, keepdim=True))
        if st["grad_total"] is not None:
            gx = gx + st["grad_total"].float()
        return {"grad_x": gx.to(t), "grad_weight": (gy * xhat).sum(0).to(st["weight"].dtype)}
    t = st["x"].dtype
    s = st["x"].float()
    out = {}
    if st["residual"] is not None:
        s = s + st["residual"].float()
        out["total"] = s.to(t)
    rstd = 1 / torch.sqrt((s * s).mean(1) + EPS)
    y = s * rstd[:, None] * w
    if c["out"] == "f8":
        scale = y.abs().amax(1) / F8_MAX
        q = torch.where(scale[:, None] > 0, y / scale[:, None], y).clamp(-F8_MAX, F8_MAX)
        out["y"], out["scale"] = q.to(torch.float8_e4m3fn), scale
    else:
        out["y"], out["rstd"] = y.to(t), rstd
    return out


TEACHER_TEMPERATURE = 0.05


def _plain_distill(st):
    c = st["case"]
    T = c["temperature"]
    z = st["logits"].float()
    here = torch.gather(z, 1, st["best"].clamp_min(0))
    t = st["scores"].masked_fill((st["best"] < 0) | (here == -math.inf), -math.inf) / TEACHER_TEMPERATURE
    live = (t > -math.inf).any(1) & (st["weight"] != 0)
    zm = z.amax(1, keepdim=True).clamp_min(-3.4e38)
    e = torch.exp((z - zm) / T)
    total = e.sum(1, keepdim=True)
    tm = t.amax(1, keepdim=True).clamp_min(-3.4e38)
    te = torch.exp(t - tm)
    tt = te.sum(1, keepdim=True)
    p = te / tt
    log_q = (here - zm) / T - torch.log(total)
    log_p = (t - tm) - torch.log(tt)
    terms = torch.where(p > 0, p * (log_p - log_q), torch.zeros_like(p))
    loss = torch.where(live, st["weight"] * T * T * terms.sum(1), torch.zeros_like(st["weight"]))
    grad = (e / total).scatter_add(1, st["best"].clamp_min(0), -p)
    scale = torch.where(live, st["weight"] * st["grad_loss"] * T, torch.zeros_like(st["weight"]))
    grad = torch.where(live[:, None], grad * scale[:, None], torch.zeros_like(grad))
    return {"loss": loss, "grad_logits": grad.to(st["logits"].dtype)}


# ---------------------------------------------------------------- the library
@functools.lru_cache(maxsize=1)
def _handle():
    import sparse_embedding_exact_gb300 as sec

    return sec.SparseCosine(65_536, chunk_rows=256)


def _own(st):
    h, c = _handle(), st["case"]
    if c["op"] == "linear":
        if c["grad"]:
            gx, gw, gb = h.linear_backward(st["grad_y"], st["x"], st["w"], pre=st["pre"], activation=c["act"])
            return {"grad_x": gx, "grad_w": gw, "grad_bias": gb}
        keep = c["act"] in ("gelu", "gelu_tanh", "silu")
        y = h.linear(st["x"], st["w"], bias=st["bias"], activation=c["act"], residual=st["residual"],
                     x_scale=st.get("x_scale"), w_scale=st.get("w_scale"), save_pre=keep)
        return {"y": y[0], "pre": y[1]} if keep else {"y": y}
    if c["op"] == "rms":
        if c["grad"]:
            gx, gw = h.rms_norm_backward(st["grad_y"], st["total"], st["weight"], st["rstd"],
                                         grad_total=st["grad_total"])
            return {"grad_x": gx, "grad_weight": gw}
        if c["out"] == "f8":
            y, scale, total = h.rms_norm_quantized(st["x"], st["weight"], residual=st["residual"], eps=EPS)
            out = {"y": y, "scale": scale}
        else:
            y, total, rstd = h.rms_norm(st["x"], st["weight"], residual=st["residual"], eps=EPS)
            out = {"y": y, "rstd": rstd}
        if st["residual"] is not None:
            out["total"] = total
        return out
    if c["fused"]:
        loss, grad = h.distill_step(st["logits"], st["scores"], st["best"], st["grad_loss"], weight=st["weight"],
                                    temperature=c["temperature"], teacher_temperature=TEACHER_TEMPERATURE)
    else:
        loss, stats = h.distill(st["logits"], st["scores"], st["best"], weight=st["weight"],
                                temperature=c["temperature"], teacher_temperature=TEACHER_TEMPERATURE)
        grad = h.distill_backward(st["grad_loss"], st["logits"], st["scores"], st["best"], stats,
                                  weight=st["weight"], temperature=c["temperature"],
                                  teacher_temperature=TEACHER_TEMPERATURE)
    return {"loss": loss, "grad_logits": grad}


def run(state):
    if own:
        return _own(state)
    return {"linear": _plain_linear, "rms": _plain_rms, "distill": _plain_distill}[state["case"]["op"]](state)


def work(case):
    size = {"bf16": 2, "f16": 2, "f8": 1, "f32": 4}[case["type"]]
    if case["op"] == "linear":
        m, k, n = case["m"], case["k"], case["n"]
        wide = max(size, 2)
        if case["grad"]:  # grad_y, pre, x, w in; grad_x, grad_w, grad_bias out
            b = 2 * (m * k + n * k) * size + m * n * size * (1 if case["act"] == "none" else 2) + 4 * n
            return {"bytes": b, "flops": 4 * m * n * k}
        outs = 1 + (case["act"] in ("gelu", "gelu_tanh", "silu")) + bool(case["residual"])
        b = (m * k + n * k) * size + m * n * wide * outs + 4 * n + (4 * (m + n) if size == 1 else 0)
        return {"bytes": b, "flops": 2 * m * n * k}
    if case["op"] == "rms":
        e = case["rows"] * case["cols"]
        if case["grad"]:
            return {"bytes": e * size * (4 if case["residual"] else 3) + 2 * case["cols"] * size + 4 * case["rows"],
                    "flops": 10 * e}
        b = e * size * (3 if case["residual"] else 1) + e * (1 if case["out"] == "f8" else size)
        return {"bytes": b + case["cols"] * size + 4 * case["rows"], "flops": 6 * e}
    e = case["rows"] * case["items"]
    return {"bytes": 2 * e * size + case["rows"] * (case["k"] * (8 + 4) + 12), "flops": 8 * e}


# ------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    d = torch.float64
    if case["op"] == "linear":
        x, w = st["x"].to(d), st["w"].to(d)
        if case["type"] == "f8":
            x = x * st["x_scale"].to(d).unsqueeze(1)
            w = w * st["w_scale"].to(d).unsqueeze(1)
        name = case["act"]
        act = {"none": lambda z: z, "relu": torch.relu, "gelu": torch.nn.functional.gelu,
               "gelu_tanh": lambda z: torch.nn.functional.gelu(z, approximate="tanh"),
               "silu": torch.nn.functional.silu, "log1p_relu": lambda z: torch.relu(z).log1p()}[name]
        if case["grad"]:
            z = st["pre"].to(d).requires_grad_()
            gz, = torch.autograd.grad(act(z), z, st["grad_y"].to(d))
            return {"grad_x": torch.mm(gz, w), "grad_w": torch.mm(gz.t(), x), "grad_bias": gz.sum(0)}
        z = torch.addmm(st["bias"].to(d), x, w.t())
        y = act(z) if st["residual"] is None else act(z) + st["residual"].to(d)
        return {"y": y, "pre": z} if name in ("gelu", "gelu_tanh", "silu") else {"y": y}
    if case["op"] == "rms":
        if case["grad"]:
            s, w = st["total"].to(d).requires_grad_(), st["weight"].to(d)
            gy, rstd, n = st["grad_y"].to(d), st["rstd"].to(d)[:, None], case["cols"]
            with torch.no_grad():
                dot = torch.einsum("rc,rc,c->r", gy, s, w)[:, None]
                gx = rstd * gy * w - s * rstd ** 3 * dot / n
                if st["grad_total"] is not None:
                    gx += st["grad_total"].to(d)
                gw = torch.einsum("rc,rc,r->c", gy, s, rstd[:, 0])
            return {"grad_x": gx.detach(), "grad_weight": gw.detach()}
        s, out = st["x"].to(d), {}
        if st["residual"] is not None:
            s = s + st["residual"].to(d)
            out["total"] = s
        rstd = (torch.linalg.vector_norm(s, dim=1) ** 2 / case["cols"] + EPS) ** -0.5
        y = s * torch.outer(rstd, st["weight"].to(d))
        if case["out"] == "f8":
            scale = torch.linalg.vector_norm(y, ord=math.inf, dim=1) / F8_MAX
            q = y / scale[:, None]
            # to the nearest value of 3 bits after the point, 2^-9 the smallest
            unit = torch.exp2(torch.floor(torch.log2(q.abs().clamp_min(2.0 ** -6))) - 3)
            return dict(out, y=torch.round(q / unit) * unit, scale=scale)
        return dict(out, y=y, rstd=rstd)
    T, rows = case["temperature"], case["rows"]
    loss = torch.zeros(rows, dtype=d, device="cuda")
    grad = torch.zeros((rows, case["items"]), dtype=d, device="cuda")
    part = max(1, 100_000_000 // case["items"])
    for a in range(0, rows, part):
        b = min(rows, a + part)
        z = st["logits"][a:b].to(d)
        best, score, weight = st["best"][a:b], st["scores"][a:b].to(d), st["weight"][a:b].to(d)
        dead = (best < 0) | (torch.take_along_dim(z, best.clamp_min(0), 1) == -math.inf)
        score = torch.where(dead, torch.full_like(score, -math.inf), score)
        ok = (~dead).any(1) & (weight != 0)
        log_p = torch.log_softmax(torch.where(ok[:, None], score, torch.zeros_like(score)) / TEACHER_TEMPERATURE, 1)
        log_q = torch.log_softmax(z / T, 1)
        p = torch.where(ok[:, None], log_p.exp(), torch.zeros_like(log_p))
        at = torch.take_along_dim(log_q, best.clamp_min(0), 1)
        kl = torch.where(p > 0, p * (log_p - at), torch.zeros_like(p)).sum(1)
        loss[a:b] = torch.where(ok, weight * T ** 2 * kl, torch.zeros_like(kl))
        q = log_q.exp()
        q.scatter_add_(1, best.clamp_min(0), -p)
        q *= (weight * st["grad_loss"][a:b].to(d) * T)[:, None]
        grad[a:b] = torch.where(ok[:, None], q, torch.zeros_like(q))
    return {"loss": loss, "grad_logits": grad}
