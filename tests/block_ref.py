"""The operators around the product, from their definitions in 64 bits, with
what single precision may change in each result.

Every function returns, beside a result, a bound on the error of a computation
of the same formula in float32 (U = 2^-24, half a step), counted operation by
operation, before the result is rounded to its own type; rounded() adds that.
Sums of n terms by any order in which no term passes more than d additions are
off by at most d U times the sum of the terms' magnitudes.
"""
import math

import torch

U = 2.0 ** -24
TINY = 1e-37          # below the smallest normal float32 a product may lose all its bits
GELU_A, GELU_B = 2.0 * math.sqrt(2.0 / math.pi), 0.044715


def rounded(x, tol, dtype):
    """The bound of x once it is rounded to dtype (float32 counts its own rounding in tol)."""
    return tol if dtype == torch.float32 else tol + (torch.finfo(dtype).eps / 2) * (x.abs() + tol) + 1e-39


def depth(n):
    """Additions that a term of a row sum passes: at most n / 64 in its lane, then a tree."""
    return math.ceil(n / 64) + 16


def norm(h, gain, eps):
    """rstd [R], y [R][C] of h (float64) and their bounds (relative for rstd)."""
    C = h.shape[1]
    ms = h.square().sum(1) / C + eps
    rstd = 1 / ms.sqrt()
    rel = (0.5 * (depth(C) + 4) + 4) * U
    y = h * rstd[:, None] * gain
    return rstd, rel, y, y.abs() * (rel + 3 * U) + TINY


def norm_backward(dy, h, gain, rstd, dH):
    C = h.shape[1]
    xhat, t = h * rstd[:, None], dy * gain
    mean = (t * xhat).sum(1, keepdim=True) / C
    dx = rstd[:, None] * (t - xhat * mean)
    e_mean = (depth(C) + 4) * U * (t * xhat).abs().sum(1, keepdim=True) / C
    e = rstd[:, None] * (4 * U * t.abs() + xhat.abs() * (e_mean + 5 * U * mean.abs())) + 2 * U * dx.abs()
    if dH is not None:
        dx = dx + dH
        e = e + U * dx.abs()
    g = dy * xhat
    return dx, e + TINY, g.sum(0), (g.shape[0] + 4) * U * g.abs().sum(0) + TINY


def _sigmoid_argument(z, act):
    if act == "silu":
        return z, torch.ones_like(z)
    return GELU_A * (z + GELU_B * z ** 3), GELU_A * (1 + 3 * GELU_B * z * z)


def activation(z, ez, act):
    """act(z) and its bound for z known to within ez."""
    if act == "none":
        return z, ez
    if act == "relu":
        return z.clamp_min(0), ez
    if act == "relu2":
        p = z.clamp_min(0)
        return p * p, 2 * p * ez + ez * ez + U * p * p
    u, _ = _sigmoid_argument(z, act)
    y = z * torch.sigmoid(u)
    # exp(-u): u off by 4 roundings, the power by 2 more; the reciprocal, the sum and the product 5
    return y, 1.2 * ez + y.abs() * (4 * u.abs() + 8) * U + TINY * (1 + z.abs())


def slope(z, act):
    """act'(z) and its bound."""
    if act == "none":
        return torch.ones_like(z), torch.zeros_like(z)
    if act == "relu":
        return (z > 0).double(), torch.zeros_like(z)
    if act == "relu2":
        return 2 * z.clamp_min(0), torch.zeros_like(z)
    u, du = _sigmoid_argument(z, act)
    p, q = torch.sigmoid(u), torch.sigmoid(-u)
    rel = (4 * u.abs() + 8) * U
    d = p + z * p * q * du
    return d, p * rel + (z * p * q * du).abs() * (2 * rel + 10 * U) + 2 * U * d.abs() + 1e-30


def epilogue_backward(dy, z, act):
    s, es = slope(z, act)
    dz = dy * s
    e = dy.abs() * es + U * dz.abs() + TINY
    return dz, e, dz.sum(0), e.sum(0) + (dz.shape[0] + 4) * U * dz.abs().sum(0)


def unpack(Wp):
    """Stored codes [N][K/4] -> weights [N][K] as float64."""
    codes = torch.stack([(Wp >> (2 * i)) & 3 for i in range(4)], 2).reshape(Wp.shape[0], -1).double()
    return (codes == 1).double() - (codes == 2).double()


def product(A, Wp, rs, ws, bias, act, res):
    acc = A.double() @ unpack(Wp).t()           # whole numbers below 2^53: exact
    s = acc * rs.double()[:, None] * ws
    z, ez = s, 3 * U * s.abs() + TINY
    if bias is not None:
        z = s + bias.double()
        ez = ez + U * z.abs()
    y, ey = activation(z, ez, act)
    if res is not None:
        y = y + res.double()
        ey = ey + U * y.abs()
    return z, ez, y, ey


def int8_rows(y, e):
    """The scale max|y| / 127 of each row and its bound."""
    s = y.abs().amax(1) / 127
    return s, (e.amax(1) / 127 + 2 * U * s) + 1e-44


def check(got, want, tol, what):
    got = got.double()
    bad = ~((got - want).abs() <= tol)
    if bool(bad.any()):
        i = tuple(int(v) for v in bad.nonzero()[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {i}: {float(got[i])!r} for "
                             f"{float(want[i])!r}, bound {float(tol.expand_as(want)[i]):.3g}")


def check_int8(Q, scale, y, e, what):
    """Q and scale stand for y, known to within e: the scale by its own bound, each value to half a step."""
    s, es = int8_rows(y, e)
    check(scale, s, es, f"{what}: scale")
    step = scale.double()[:, None]
    # the quotient is rounded once (at most 127 U) before it goes to a whole number; 127.0000x is held at 127
    check(Q.double() * step, y, step * (0.5 + 130 * U) + e + 127 * es[:, None], f"{what}: int8 values")
    assert int(Q.abs().max()) <= 127
