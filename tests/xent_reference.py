"""The cross entropy over every item in 64 bits, on whatever device the inputs
are, for the tests: the formulas written out, one rounding nowhere; and the
bounds of what the float32 kernels may be off."""
import math

import torch

from dense_reference import F64, ROUND, STEP

E = 2.0 ** -24


def cross_entropy(x, w, targets, grad_loss=None, bias=None, weight=None, temperature=1.0):
    """A dict of loss, grad_x, grad_w, grad_bias, gz and live (the rows that
    are not absent)."""
    M, V = x.shape[0], w.shape[0]
    one = torch.ones(M, dtype=F64, device=x.device)
    wt = one if weight is None else weight.to(F64)
    g = one if grad_loss is None else grad_loss.to(F64)
    inside = (targets >= 0) & (targets < V) & (wt != 0)
    xs = torch.where(inside[:, None], x.to(F64), torch.zeros((), dtype=F64, device=x.device))
    z = xs @ w.to(F64).t()
    if bias is not None:
        z = z + bias.to(F64)
    z = z / temperature
    at = targets.clamp(0, V - 1)[:, None]
    here = z.gather(1, at)[:, 0]
    live = inside & (here != -math.inf)
    z = torch.where(live[:, None], z, torch.zeros_like(z))
    here = z.gather(1, at)[:, 0]
    lse = torch.logsumexp(z, 1)
    loss = torch.where(live, wt * (lse - here), torch.zeros_like(here))
    p = torch.exp(z - lse[:, None])
    hot = torch.zeros_like(z).scatter_(1, at, 1.0)
    scale = torch.where(live, wt * g / temperature, torch.zeros_like(here))
    gz = torch.where(live[:, None], (p - hot) * scale[:, None], torch.zeros_like(p))
    xl = torch.where(live[:, None], xs, torch.zeros_like(xs))
    return {"loss": loss, "grad_x": gz @ w.to(F64), "grad_w": gz.t() @ xl, "grad_bias": gz.sum(0), "gz": gz, "live": live,
            "z": z, "p": p, "hot": hot, "scale": scale, "x": xl}


def sum_bound(size, k):
    """Of a float32 sum of k exact products on the tensor cores: a partial sum
    of size S is rounded (or cut) once for each 16 of them, the tree within them
    and the shares of a cluster, at most 2^-23 S each; then bias and scales."""
    return (k / 16 + 24) * 2.0 ** -23 * size


def bounds(r, x, w, bias=None, weight=None, grad_loss=None, temperature=1.0, dtype=None, pieces=1):
    """How far the kernels' outputs may be from `r`, cross_entropy()'s of the
    same arguments.  A logit is off by its sum's bound.  An exponent's argument
    (log2 e / T times logit minus base) is off by three roundings relative to
    itself, ex2 by 2^-22; a row's sum of V of them is added up in chains of at
    most V / 7 + 64 roundings, rescalings included; the softmax has both twice.
    The softmax less its target is then rounded to x's type (that of binary16
    times 2^14: half a step 2^-39), and for grad_w x times its row's factor
    (that of binary16 times a power of two that brings the largest factor to
    1/2 at least: half a step at most 2^-24 of that)."""
    V, K = w.shape
    size = r["x"].abs() @ w.to(F64).abs().t()
    if bias is not None:
        size = size + torch.where(torch.isinf(bias), torch.zeros_like(bias), bias).to(F64).abs()
    off_z = sum_bound(size, K) / temperature
    finite = torch.isfinite(r["z"])
    big = torch.where(finite, r["z"], torch.full_like(r["z"], -math.inf)).amax(1)
    low = torch.where(finite, r["z"], torch.full_like(r["z"], math.inf)).amin(1)
    reach = (big - low).clamp_min(0) * 1.45
    worst = off_z.amax(1)
    off_sum = worst + 3 * E * reach + (V / 7 + 64) * E
    at_hot = (off_z * r["hot"]).sum(1)
    wt = 1.0 if weight is None else weight.to(F64).abs()
    loss = torch.where(r["live"], wt * (off_sum + at_hot + 8 * E * (1 + reach + r["loss"].abs())), torch.zeros_like(r["loss"]))
    s = r["scale"].abs()[:, None]
    rel = 2 * (off_sum[:, None] + off_z)
    # an exponential below 2^-126 is 0 (ex2 flushes it), and is divided by a sum
    # of 1 at least: 2^-126 |scale| more
    soft = s * r["p"] * rel + 4 * E * s * (r["p"] + r["hot"]) + s * 2.0 ** -126
    top = float(s.max()) if s.numel() else 0.0
    half = s * (2.0 ** -39 if x.dtype == torch.float16 else STEP[x.dtype])
    off = soft + ROUND[x.dtype] * (r["gz"].abs() + soft) + torch.where(r["live"][:, None], half, torch.zeros_like(half))
    full = r["gz"].abs() + off
    M = x.shape[0]
    wa, xa = w.to(F64).abs(), r["x"].abs()
    # the rounding of a row of x times its factor, in that product's terms
    unit = torch.where(s > 0, full / s.clamp_min(1e-300), torch.zeros_like(full))
    step_x = 2.0 ** -24 * top if x.dtype == torch.float16 else STEP[x.dtype]
    off_x = ROUND[x.dtype] * full.t() @ xa + unit.t() @ torch.full_like(xa, step_x)
    out = dtype or x.dtype
    close = lambda want, extra: ROUND[out] * (want.abs() + extra) + extra + STEP[out]  # noqa: E731
    gx = close(r["grad_x"], off @ wa + sum_bound(full @ wa, V) + pieces * E * (full @ wa))
    gw = close(r["grad_w"], (1 + ROUND[x.dtype]) * (off.t() @ xa) + off_x + sum_bound(full.t() @ xa + off_x, M))
    gb = soft.sum(0) + (64 + M / 8) * E * full.sum(0) + 2.0 ** -149
    return {"loss": loss + 2.0 ** -149, "grad_x": gx, "grad_w": gw, "grad_bias": gb}
