"""The training operators' definitions in 64 bits, on any device, written from
their formulas (none of the library's code)."""
from __future__ import annotations

import math

import torch

F64 = torch.float64


def spans(offsets):
    o = [int(v) for v in offsets]
    return list(zip(o[:-1], o[1:]))


def dgrad(dout, offsets, w):
    out = torch.zeros((dout.shape[0], w.shape[2]), dtype=F64, device=dout.device)
    for e, (a, b) in enumerate(spans(offsets)):
        out[a:b] = dout[a:b].to(F64) @ w[e].to(F64)
    return out


def wgrad(dout, offsets, x, E):
    out = torch.zeros((E, dout.shape[1], x.shape[1]), dtype=F64, device=dout.device)
    for e, (a, b) in enumerate(spans(offsets)):
        out[e] = dout[a:b].to(F64).t() @ x[a:b].to(F64)
    return out


def round8(x):
    """(values the 8-bit form stands for, scale exponents q) of x [R, c]: found by trying, not by bit arithmetic.

    Every block of 32 gets the first power of two of -124, -123, ... that brings its largest finite
    magnitude to 448 or below, every value the nearest of the format's non-negative values (ties to
    the even code) with its sign."""
    codes = torch.arange(127, dtype=torch.int64)  # 0x00 .. 0x7e; 0x7f is NaN
    e, m = codes >> 3, codes & 7
    values = torch.where(e == 0, m.to(F64) * 2.0 ** -9, (1 + m.to(F64) / 8) * torch.pow(2.0, (e - 7).to(F64)))
    assert float(values.max()) == 448.0
    R, c = x.shape
    b = x.detach().cpu().to(F64).view(R * c // 32, 32)
    finite = torch.isfinite(b)
    big = torch.where(finite, b.abs(), torch.zeros_like(b)).amax(1)
    q = torch.full((b.shape[0],), -124, dtype=torch.int64)
    while True:
        over = big > 448.0 * torch.pow(2.0, q.to(F64))
        if not bool(over.any()):
            break
        q += over.to(torch.int64)
    scale = torch.pow(2.0, q.to(F64))[:, None]
    z = torch.where(finite, b.abs(), torch.zeros_like(b)) / scale
    hi = torch.searchsorted(values, z).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    dlo, dhi = z - values[lo], values[hi] - z
    pick = torch.where((dlo < dhi) | ((dlo == dhi) & (lo % 2 == 0)), lo, hi)
    v = torch.copysign(values[pick], b) * scale
    v = v.clamp(-1.875 * 2.0 ** 127, 1.875 * 2.0 ** 127)  # finite values stay finite in bf16
    v = torch.where(finite, v, torch.full_like(v, math.nan))
    return v.view(R, c), q.view(R, c // 32)


def swiglu(g, u):
    g, u = g.to(F64), u.to(F64)
    return g * torch.special.expit(g) * u


def swiglu_bwd(dh, g, u, w):
    """dgate, dup, hw, drow_weight for the values g, u [S, f] that the checkpoint holds."""
    dh, g, u, w = dh.to(F64), g.to(F64), u.to(F64), w.to(F64)[:, None]
    s = torch.special.expit(g)
    a = g * s
    return w * dh * u * (s + a * (1 - s)), w * dh * a, w * a * u, (dh * a * u).sum(1)


def layernorm(x, gamma, beta, eps):
    x = x.to(F64)
    mean = x.mean(1, keepdim=True)
    rstd = 1 / torch.sqrt(((x - mean) ** 2).mean(1, keepdim=True) + eps)
    return (x - mean) * rstd * gamma.to(F64) + beta.to(F64), mean[:, 0], rstd[:, 0]


def layernorm_bwd(dy, x, gamma, eps, dres=None):
    _, mean, rstd = layernorm(x, gamma, torch.zeros_like(gamma), eps)
    dy, xh = dy.to(F64), (x.to(F64) - mean[:, None]) * rstd[:, None]
    t = dy * gamma.to(F64)
    dx = rstd[:, None] * (t - t.mean(1, keepdim=True) - xh * (t * xh).mean(1, keepdim=True))
    if dres is not None:
        dx = dx + dres.to(F64)
    return dx, (dy * xh).sum(0), dy.sum(0)
