"""Values kept in 8 bits, in 64 bits and on whatever device the inputs are, for
the tests: the format written out."""
import math

import torch

from dense_reference import F64

GROUP = 32
LEAST = {torch.float32: -126, torch.bfloat16: -124, torch.float16: -15}
LARGEST = {t: torch.finfo(t).max for t in LEAST}


def _groups(x):
    """(rows, groups, 32), short groups filled with zeros."""
    rows, cols = x.shape
    n = (cols + GROUP - 1) // GROUP
    full = torch.zeros((rows, n * GROUP), dtype=x.dtype, device=x.device)
    full[:, :cols] = x
    return full.view(rows, n, GROUP)


def exponents(x, least):
    """The smallest e with max|x| <= 448 2^e over each group's finite values."""
    g = _groups(x.to(F64))
    most = torch.where(torch.isfinite(g), g.abs(), torch.zeros_like(g)).amax(2)
    mantissa, e = torch.frexp(most / 448)  # most = mantissa 448 2^e, mantissa in [1/2, 1)
    e = e - (mantissa == 0.5).int()
    return torch.where(most > 0, e, torch.full_like(e, least)).clamp_min(least)


def codes(x, e):
    """The nearest e4m3 values of x 2^-e (ties to even), NaN where x is not finite."""
    cols = x.shape[1]
    q = _groups(x.to(F64)) * torch.exp2(-e.to(F64))[:, :, None]
    unit = torch.exp2(torch.floor(torch.log2(q.abs().clamp_min(2.0 ** -6).nan_to_num(1.0, posinf=1.0))) - 3)
    r = torch.round(q / unit) * unit
    r = torch.where(torch.isfinite(q), r, torch.full_like(r, math.nan))
    return r.flatten(1)[:, :cols]


def values(q, e):
    """What codes (as numbers) and exponents stand for."""
    return (_groups(q.to(F64)) * torch.exp2(e.to(F64))[:, :, None]).flatten(1)[:, :q.shape[1]]


def exponents_of(scale):
    return scale.view(torch.uint8).to(torch.int32) - 127


def compressed(x):
    """(codes as numbers, exponents, values) of a matrix."""
    e = exponents(x, LEAST[x.dtype])
    q = codes(x, e)
    return q, e, values(q, e)


def stand_for(q, scale, dtype=None):
    """The values of codes and scales, beyond the type's largest that."""
    v = values(q.to(F64), exponents_of(scale))
    return v if dtype is None else v.clamp(-LARGEST[dtype], LARGEST[dtype])
