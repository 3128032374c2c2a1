"""The layer operators' formulas in 64 bits, and how far a result that holds
its sums in binary32 and rounds once may be from them.

A sum of k products in binary32 is off by at most (k + 2) * 2^-24 of the sum
of the magnitudes in any order, and twice that where a matrix unit truncates;
an activation computed in binary32 by at most 2^-20 of 1 + |z| (a dozen
roundings, slopes below 1.2); a rounding to type t by half a step,
finfo(t).eps / 2 of the value, or half the least subnormal.
"""

import math

import torch


def act_pair(name, z):
    """act(z) and act'(z) in 64 bits."""
    if name == "relu":
        return z.clamp_min(0), (z > 0).to(z.dtype)
    if name == "silu":
        s = torch.sigmoid(z)
        return z * s, s * (1 + z * (1 - s))
    if name == "gelu":
        c = 0.5 * torch.erfc(-z / math.sqrt(2))
        return z * c, c + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        q = math.sqrt(2 / math.pi)
        t = torch.tanh(q * (z + 0.044715 * z ** 3))
        return 0.5 * z * (1 + t), 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * q * (1 + 3 * 0.044715 * z * z)
    return z, torch.ones_like(z)


def rounding(dtype, value):
    """Half a step of `dtype` at `value`."""
    fi = torch.finfo(dtype)
    return fi.eps / 2 * value.abs() + fi.smallest_normal * fi.eps / 2


def sum_error(k, magnitudes):
    return (k + 2) * 2.0 ** -23 * magnitudes


def act_error(z, dz):
    """Of act(z) or act'(z) for a z that is off by dz: slopes and curvatures below 1.2."""
    return 1.2 * dz + 2.0 ** -20 * (1 + z.abs())


def linear(x, w, bias, residual, act, k):
    """(y, its error before rounding, z, its error) for 64-bit inputs."""
    z, mag = x @ w.t(), x.abs() @ w.abs().t()
    if bias is not None:
        z, mag = z + bias, mag + bias.abs()
    ez = sum_error(k + 1, mag)
    y = act_pair(act, z)[0]
    ey = ez if act == "none" else act_error(z, ez)
    if residual is not None:
        y = y + residual
        ey = ey + 2.0 ** -23 * (y.abs() + residual.abs())
    return y, ey, z, ez


def product(a, b, ea, terms):
    """a b for a that is off by ea, in binary32 sums."""
    return a @ b, ea @ b.abs() + sum_error(terms, (a.abs() + ea) @ b.abs())


def slope(dy, pre, act, dtype):
    """(dz, its error before rounding, its error after rounding to dtype)."""
    if act == "none":
        return dy, torch.zeros_like(dy), torch.zeros_like(dy)
    s = act_pair(act, pre)[1]
    dz = dy * s
    e = dy.abs() * act_error(pre, 0.0) + 2.0 ** -23 * dz.abs()
    return dz, e, e + rounding(dtype, dz.abs() + e)


def check(name, got, want, error, dtype):
    assert got.dtype == dtype, (name, got.dtype)
    tol = error + rounding(dtype, want.abs() + error)
    off = (got.double() - want).abs()
    bad = ~(off <= tol)
    assert not bool(bad.any()), (name, tuple(got.shape), int(bad.sum()), float((off - tol).max()),
                                 bad.nonzero()[0].tolist())
