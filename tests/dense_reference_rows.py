"""The 64-bit form of the distillation for many rows at once (dense_reference's
takes a row at a time): the same outputs and bounds."""
import math

import torch

F64 = torch.float64


def distill(logits, scores, items, weight=None, grad_loss=None, temperature=1.0, teacher_temperature=1.0):
    """(loss, grad, bound of the loss's terms, room of the gradient's terms)."""
    R, V = logits.shape
    one = torch.ones(R, dtype=F64, device=logits.device)
    w = one if weight is None else weight.to(F64)
    g = one if grad_loss is None else grad_loss.to(F64)
    z = logits.to(F64)
    at = items.clamp(0, V - 1)
    here = z.gather(1, at)
    absent = (items < 0) | (items >= V) | (scores == -math.inf) | (here == -math.inf)
    live = (~absent).any(1) & (w != 0)
    zero = torch.zeros((), dtype=F64, device=logits.device)
    # rows that are not live get harmless values, and zeros at the end
    t = torch.where(absent, torch.full_like(here, -math.inf), scores.to(F64) / teacher_temperature)
    t = torch.where(live[:, None], t, zero)
    t = t - t.amax(1, keepdim=True)
    log_p = t - torch.logsumexp(t, 1, keepdim=True)
    p = torch.where(live[:, None], log_p.exp(), zero)
    x = torch.where(live[:, None], z, zero)
    x = (x - x.amax(1, keepdim=True)) / temperature
    log_s = torch.log(torch.exp(x).sum(1, keepdim=True))
    q = torch.exp(x - log_s)
    xj = x.gather(1, at)
    have = p > 0
    T2 = temperature ** 2
    kl = torch.where(have, p * (log_p - (xj - log_s)), zero).sum(1)
    size = torch.where(have, p * (1 + log_p.abs() + xj.abs() + log_s), zero).sum(1)
    scale = (w * g * temperature)[:, None]
    grad = (scale * q).scatter_add_(1, at, -scale * p)
    far = torch.where(x > -math.inf, x.abs() + 16, zero)
    tj = torch.where(absent, zero, t.abs())
    room = (scale.abs() * q * far).scatter_add_(1, at, scale.abs() * p * (16 + tj))
    dead = ~live
    return ((w * T2 * kl).masked_fill(dead, 0), grad.masked_fill_(dead[:, None], 0),
            (w.abs() * T2 * size).masked_fill(dead, 0), room.masked_fill_(dead[:, None], 0))
