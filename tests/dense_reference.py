"""Plain 64-bit forms of the dense operators, on whatever device the inputs
are, for the tests: the formulas written out, one rounding nowhere."""
import math

import torch

F64 = torch.float64
# Unit roundoff of each type, and half its smallest step.
ROUND = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
STEP = {torch.float32: 2.0 ** -149, torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -25}


def rms_norm(x, weight, residual=None, eps=1e-6):
    s = x.to(F64) if residual is None else x.to(F64) + residual.to(F64)
    rstd = 1 / torch.sqrt((s * s).mean(1) + eps)
    return s * rstd[:, None] * weight.to(F64), s, rstd


def rms_norm_grad(grad_y, total, weight, rstd, grad_total=None):
    gy, xh = grad_y.to(F64), total.to(F64) * rstd.to(F64)[:, None]
    g = gy * weight.to(F64)
    gx = rstd.to(F64)[:, None] * (g - xh * (g * xh).mean(1, keepdim=True))
    if grad_total is not None:
        gx = gx + grad_total.to(F64)
    return gx, (gy * xh).sum(0)


def act(z, name):
    if name == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if name == "gelu":
        return z * 0.5 * torch.erfc(-z / math.sqrt(2))
    if name == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    if name == "silu":
        return z / (1 + torch.exp(-z))
    if name == "log1p_relu":
        return torch.log1p(torch.where(z > 0, z, torch.zeros_like(z)))
    return z


def act_grad(z, name):
    """d act / dz, 0 at the kink of the rectified ones."""
    if name in ("none",):
        return torch.ones_like(z)
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "gelu":
        return 0.5 * torch.erfc(-z / math.sqrt(2)) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z ** 3))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)
    if name == "silu":
        s = 1 / (1 + torch.exp(-z))
        return s * (1 + z * (1 - s))
    return torch.where(z > 0, 1 / (1 + torch.where(z > 0, z, torch.zeros_like(z))), torch.zeros_like(z))


def linear(x, w, bias=None, activation="none", residual=None, x_scale=None, w_scale=None):
    """(y, pre, sum of |products| that z adds up)."""
    a, b = x.to(F64), w.to(F64)
    if x_scale is not None:
        a, b = a * x_scale.to(F64)[:, None], b * w_scale.to(F64)[:, None]
    z = a @ b.t()
    size = a.abs() @ b.abs().t()
    if bias is not None:
        z = z + bias.to(F64)
        size = size + bias.to(F64).abs()
    y = act(z, activation)
    return (y if residual is None else y + residual.to(F64)), z, size


def linear_grad(grad_y, x, w, pre=None, activation="none"):
    gz = grad_y.to(F64)
    if activation != "none":
        gz = gz * act_grad(pre.to(F64), activation)
    return gz @ w.to(F64), gz.t() @ x.to(F64), gz.sum(0), gz


def distill(logits, scores, items, weight=None, grad_loss=None, temperature=1.0, teacher_temperature=1.0):
    """(loss, grad, bound of the loss's terms, q, p of each entry, t of each entry)."""
    R, V = logits.shape
    loss = torch.zeros(R, dtype=F64, device=logits.device)
    terms = torch.zeros(R, dtype=F64, device=logits.device)
    grad = torch.zeros((R, V), dtype=F64, device=logits.device)
    room = torch.zeros((R, V), dtype=F64, device=logits.device)  # the gradient's terms, with their arguments' sizes
    for r in range(R):
        w = 1.0 if weight is None else float(weight[r])
        g = 1.0 if grad_loss is None else float(grad_loss[r])
        z = logits[r].to(F64)
        have = [j for j in range(scores.shape[1])
                if 0 <= int(items[r, j]) < V and float(scores[r, j]) != -math.inf
                and float(z[int(items[r, j])]) != -math.inf]
        if w == 0 or not have:
            continue
        at = items[r, have]
        t = scores[r, have].to(F64) / teacher_temperature
        t = t - t.max()
        log_p = t - torch.log(torch.exp(t).sum())
        p = torch.exp(log_p)
        x = (z - z.max()) / temperature
        log_s = torch.log(torch.exp(x).sum())
        q = torch.exp(x - log_s)
        loss[r] = w * temperature ** 2 * torch.where(p > 0, p * (log_p - (x[at] - log_s)), torch.zeros_like(p)).sum()
        terms[r] = abs(w) * temperature ** 2 * (p * (1 + log_p.abs() + x[at].abs() + log_s)).nan_to_num(0.0).sum()
        scale = w * g * temperature
        grad[r] = (scale * q).index_add(0, at, -scale * p)
        far = torch.where(x > -math.inf, x.abs() + 16, torch.zeros_like(x))
        room[r] = (abs(scale) * q * far).index_add(0, at, abs(scale) * p * (16 + t.abs()))
    return loss, grad, terms, room
