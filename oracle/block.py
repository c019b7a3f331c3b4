"""The operators around the linear layer in float64 (torch, any device): the
plain definitions that the norm, epilogue and clipping kernels are compared
with.  Inputs of any floating type are widened first; nothing is rounded."""

from __future__ import annotations

import math

import torch


def norm_fwd(x, gamma=None, beta=None, eps=1e-5, rms=False):
    """(y, mean, rstd) of each row of x; mean is None for rms."""
    x = x.double()
    mean = None if rms else x.mean(1)
    d = x if rms else x - mean[:, None]
    rstd = 1.0 / torch.sqrt((d * d).mean(1) + eps)
    y = d * rstd[:, None]
    y = y if gamma is None else y * gamma.double()
    return y if beta is None else y + beta.double(), mean, rstd


def norm_bwd(dy, x, gamma, mean, rstd, dres=None, rms=False):
    """(dx, dgamma, dbeta) for given statistics; dbeta is None for rms."""
    x, dy, rstd = x.double(), dy.double(), rstd.double()[:, None]
    xh = (x if rms else x - mean.double()[:, None]) * rstd
    g = dy if gamma is None else dy * gamma.double()
    dx = g - xh * (g * xh).mean(1, keepdim=True)
    dx = dx if rms else dx - g.mean(1, keepdim=True)
    dx = dx * rstd
    dx = dx if dres is None else dx + dres.double()
    return dx, (dy * xh).sum(0), None if rms else dy.sum(0)


def act(z, which):
    """The activations of include/falqon.h by number."""
    z = z.double()
    if which == 1:
        return torch.where(z > 0, z, torch.zeros_like(z))
    if which == 2:
        return 0.5 * z * torch.erfc(-z / math.sqrt(2.0))
    if which == 3:
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3)))
    if which == 4:
        return z / (1.0 + torch.exp(-z))
    return z


def act_slope(z, which):
    z = z.double()
    if which == 1:
        return (z > 0).double()
    if which == 2:
        return 0.5 * torch.erfc(-z / math.sqrt(2.0)) + z * torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    if which == 3:
        c = math.sqrt(2.0 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z ** 3))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * c * (1.0 + 3 * 0.044715 * z * z)
    if which == 4:
        s = 1.0 / (1.0 + torch.exp(-z))
        return s + z * s * (1.0 - s)
    return torch.ones_like(z)


def decode_e4m3(codes):
    """The values of E4M3 codes (uint8), bit by bit: sign, 4 exponent bits of bias 7, 3 mantissa bits."""
    c = codes.to(torch.int64)
    e, m = (c >> 3) & 15, (c & 7).double()
    v = torch.where(e > 0, torch.exp2((e - 7).double()) * (1.0 + m / 8.0), torch.exp2(torch.full_like(m, -6.0)) * m / 8.0)
    v = torch.where((c & 127) == 127, torch.full_like(v, math.nan), v)
    return torch.where(c >= 128, -v, v)


def linear_fwd_epilogue(xq, s_x, wq, s_w, bias=None, which=0, residual=None):
    """(y, z) of the linear layer with its epilogue."""
    z = decode_e4m3(xq) @ decode_e4m3(wq).T / (float(s_x) * float(s_w))
    z = z if bias is None else z + bias.double()
    y = act(z, which)
    return y if residual is None else y + residual.double(), z


def linear_epilogue_bwd(dy, z, which):
    """(dz, dbias)."""
    dz = dy.double() * (1.0 if which == 0 else act_slope(z, which))
    return dz, dz.sum(0)


def clip_grads(grads, max_norm, factor=1.0):
    """(outs, norm, coef); a non-finite gradient voids the step: coef 0 and zeros."""
    norm = math.sqrt(sum(float((g.double() ** 2).sum()) for g in grads))
    if not math.isfinite(norm):
        return [torch.zeros_like(g, dtype=torch.float64) for g in grads], norm, 0.0
    coef = max_norm / norm if norm > max_norm else 1.0
    return [g.double() * (factor * coef) for g in grads], norm, coef
