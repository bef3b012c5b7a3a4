"""Float64 oracle of the feed-forward block in 16 bits (include/nvfp4_ffn.h), on PyTorch tensors of any device.

Written from the formulas, apart from the package: every function takes and gives float64 tensors (codes and scales
uint8) and computes one operator for one expert's rows. Test infrastructure only.
"""
from __future__ import annotations

import math

import torch


def rows8(v):
    """(codes, scales) of rows v [rows, n]: for every 32 the least 2^e, e >= -126, with max |v| <= 448 * 2^e, and the E4M3
    code nearest to v / 2^e, ties to even. Blocks that hold an infinity or NaN: scale 255, codes 0x7F."""
    b = v.unflatten(-1, (-1, 32))
    top = b.abs().amax(-1, keepdim=True)
    bad = ~torch.isfinite(b).all(-1, keepdim=True)
    fine = torch.where(bad, torch.ones_like(top), top)
    # 448 * 2^e by multiplication, so that no logarithm decides
    e = torch.ceil(torch.log2(fine.clamp(min=1e-300) / 448)).clamp(min=-126)
    e = torch.where(fine > 448 * torch.exp2(e), e + 1, e)
    e = torch.where((fine <= 448 * torch.exp2(e - 1)) & (e > -126), e - 1, e)
    q = torch.where(bad, torch.zeros_like(b), b) / torch.exp2(e)
    a = q.abs()
    step = torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0 ** -6))) - 3)
    r = torch.round(a / step) * step  # half to even
    code = torch.where(r < 2.0 ** -6, r * 2.0 ** 9, torch.zeros_like(r))
    p = torch.floor(torch.log2(r.clamp(min=2.0 ** -6)))
    code = torch.where(r >= 2.0 ** -6, (p + 7) * 8 + (r / torch.exp2(p) - 1) * 8, code)
    code = torch.where(torch.signbit(q), code + 128, code)
    code = torch.where(bad, torch.full_like(code, 127), code)
    scale = torch.where(bad, torch.full_like(e, 255), e + 127)
    return code.to(torch.uint8).flatten(-2), scale.to(torch.uint8).squeeze(-1)


def values8(codes, scales):
    """What codes and scales stand for."""
    c = codes.to(torch.int64)
    p, m = (c >> 3) & 15, (c & 7).double()
    v = torch.where(p == 0, m * 2.0 ** -9, (1 + m / 8) * torch.exp2((p - 7).double()))
    v = torch.where((c & 127) == 127, math.nan, v) * torch.where(c >= 128, -1.0, 1.0)
    s = torch.where(scales == 255, math.nan, torch.exp2(scales.double() - 127))
    return (v.unflatten(-1, (-1, 32)) * s.unsqueeze(-1)).flatten(-2)


def cdf(z):
    return 0.5 * torch.erfc(-z * math.sqrt(0.5))


def activation(z, kind):
    if kind is None:
        return z
    if kind == "relu":
        return torch.where(z < 0, torch.zeros_like(z), z)
    if kind == "silu":
        return torch.where(z == -math.inf, torch.zeros_like(z), z / (1 + torch.exp(-z)))
    return torch.where(z == -math.inf, torch.zeros_like(z), z * cdf(z))


def slope(z, kind):
    """The activation's derivative; at infinities its limits, relu's at 0: 0."""
    if kind is None:
        return torch.ones_like(z)
    if kind == "relu":
        return torch.where(torch.isnan(z), z, (z > 0).double())
    y = z.clamp(-700, 700)
    if kind == "silu":
        p = 1 / (1 + torch.exp(-y))
        return p * (1 + y * (1 - p))
    return cdf(y) + y * torch.exp(-0.5 * y * y) / math.sqrt(2 * math.pi)


def rmsnorm(s, weight, eps):
    """(y, rstd) of rows s."""
    r = 1 / torch.sqrt((s * s).mean(1) + eps)
    y = s * r.unsqueeze(1)
    return (y if weight is None else y * weight), r


def rmsnorm_backward(dy, s, weight, rstd, dsum=None):
    h = s * rstd.unsqueeze(1)
    g = dy if weight is None else dy * weight
    dx = rstd.unsqueeze(1) * (g - h * (g * h).mean(1, keepdim=True))
    return (dx if dsum is None else dx + dsum), (dy * h).sum(0)


def linear(x, w, bias=None, act=None, residual=None):
    """(y, z)."""
    z = x @ w.T
    if bias is not None:
        z = z + bias
    y = activation(z, act)
    return (y if residual is None else y + residual), z


def linear_backward(dy, x, w, z=None, act=None):
    """(dx, dw, dbias, dz)."""
    dz = dy if act is None else dy * slope(z, act)
    return dz @ w, dz.T @ x, dz.sum(0), dz


def gated(x, w, act="silu"):
    """(h, g and u side by side)."""
    z = x @ w.T
    g, u = z.chunk(2, 1)
    return activation(g, act) * u, z


def gated_dz(dh, z, act="silu"):
    g, u = z.chunk(2, 1)
    return torch.cat((dh * u * slope(g, act), dh * activation(g, act)), 1)
