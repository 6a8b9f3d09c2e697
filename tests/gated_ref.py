"""The operators of a gated block with a layer norm and 8-bit weights, from
their definitions in 64 bits, with what single precision may change in each
result; in the terms of block_ref (U, depth, activation, slope)."""
import torch

import block_ref as ref
from block_ref import TINY, U, depth


def layernorm(h, gain, beta, eps):
    """mean, rstd [R], y [R][C] of h (float64) and the bounds of each (relative for rstd)."""
    C = h.shape[1]
    mean = h.sum(1) / C
    e_mean = (depth(C) + 1) * U * h.abs().sum(1) / C + U * mean.abs() + TINY
    d = h - mean[:, None]
    e_d = e_mean[:, None] + U * d.abs()
    var = d.square().sum(1) / C
    # the squares of d off by e_d, their sum, the division and the addition of eps
    e_var = (2 * d.abs() * e_d + e_d * e_d).sum(1) / C + (depth(C) + 4) * U * (var + eps)
    rstd = 1 / (var + eps).sqrt()
    # the root of a value off by a share x is off by less than x / 2 (1 + x)
    x = e_var / (var + eps)
    rel = 0.5 * x * (1 + x) + 4 * U
    g = (rstd[:, None] * gain).abs()
    y = d * rstd[:, None] * gain
    e = g * e_d * (1 + rel[:, None]) + y.abs() * (rel[:, None] + 3 * U)
    if beta is not None:
        y = y + beta
    return mean, e_mean, rstd, rel, y, e + U * y.abs() + TINY


def layernorm_backward(dy, h, gain, mean, rstd, dH):
    R, C = h.shape
    xhat, t = (h - mean[:, None]) * rstd[:, None], dy * gain
    m1, m2 = t.sum(1, keepdim=True) / C, (t * xhat).sum(1, keepdim=True) / C
    e1 = (depth(C) + 4) * U * t.abs().sum(1, keepdim=True) / C
    e2 = (depth(C) + 8) * U * (t * xhat).abs().sum(1, keepdim=True) / C
    dx = rstd[:, None] * (t - m1 - xhat * m2)
    e = rstd[:, None] * (3 * U * t.abs() + e1 + 2 * U * m1.abs() + xhat.abs() * (e2 + 6 * U * m2.abs())) + 2 * U * dx.abs()
    if dH is not None:
        dx = dx + dH
        e = e + U * dx.abs()
    g = dy * xhat
    return (dx, e + TINY, g.sum(0), (R + 8) * U * g.abs().sum(0) + TINY, dy.sum(0), (R + 2) * U * dy.abs().sum(0) + TINY)


def gated(zg, eg, zu, eu, act):
    """act(g) u of pre-activations known to within eg, eu, and its bound."""
    a, ea = ref.activation(zg, eg, act)
    y = a * zu
    return y, ea * (zu.abs() + eu) + a.abs() * eu + U * y.abs() + TINY


def gated_product(A, Wp, rs, gate, up, bias, act):
    """(z, its bound) [M][2N] and (y, its bound) [M][N] of the ternary gated product."""
    N = Wp.shape[0] // 2
    acc = A.double() @ ref.unpack(Wp).t()
    s = acc * rs.double()[:, None]
    s = torch.cat((s[:, :N] * gate, s[:, N:] * up), 1)
    z, ez = s, 3 * U * s.abs() + TINY
    if bias is not None:
        z = s + bias.double()
        ez = ez + U * z.abs()
    return z, ez, *gated(z[:, :N], ez[:, :N], z[:, N:], ez[:, N:], act)


def gated_backward(dy, Z, act):
    """(dg | du), its bound, its column sums and their bound."""
    C = dy.shape[1]
    z, u = Z[:, :C], Z[:, C:]
    s, es = ref.slope(z, act)
    a, ea = ref.activation(z, torch.zeros_like(z), act)
    dg, du = dy * u * s, dy * a
    eg = (dy * u).abs() * (es + 2 * U * s.abs()) + 2 * U * dg.abs() + TINY * (1 + s.abs())
    eu = dy.abs() * (ea + 2 * U * a.abs()) + 2 * U * du.abs() + TINY * (1 + a.abs())
    dz, e = torch.cat((dg, du), 1), torch.cat((eg, eu), 1)
    return dz, e, dz.sum(0), e.sum(0) + (dy.shape[0] + 4) * U * dz.abs().sum(0)


def int8_product(A, W, rs, cs, bias, act, res):
    acc = A.double() @ W.double().t()           # whole numbers below 2^53: exact
    s = acc * rs.double()[:, None]
    if cs is not None:
        s = s * cs.double()
    z, ez = s, 3 * U * s.abs() + TINY
    if bias is not None:
        z = s + bias.double()
        ez = ez + U * z.abs()
    y, ey = ref.activation(z, ez, act)
    if res is not None:
        y = y + res.double()
        ey = ey + U * y.abs()
    return z, ez, y, ey
