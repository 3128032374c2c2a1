"""The token operators' formulas in 64 bits, and how far a result that holds
its sums and states in binary32 and rounds once may be from them.

U is half a step of binary32 at 1.  A sum over a row goes through at most
DEPTH additions on the way of any of its terms: 64 by one thread, 10 between
threads, and what makes the terms; so it is off by DEPTH * U of the sum of the
magnitudes.  Outputs are rounded by half a step of their type
(layer_reference.rounding)."""

import numpy as np
import torch

from layer_reference import check, rounding  # noqa: F401

U = 2.0 ** -24
DEPTH = 96


def layer_norm(x, weight, bias, eps):
    """(y, its error, mean, its error, rstd, its error) for 64-bit inputs, errors before an output's rounding.

    A mean that is off by e moves the variance by e^2 beside the sum's own error, and a variance that is off by a
    share r moves rstd by at most r, while r is below a half."""
    d = x.shape[1]
    mean = x.mean(1, keepdim=True)
    em = DEPTH * U * x.abs().sum(1, keepdim=True) / d + U * mean.abs()
    if d == 1:  # nothing is added or rounded: zeros beside the one element, divided by 1
        em = torch.zeros_like(em)
    off = x - mean
    eoff = em + U * (off.abs() + em)
    var = (off * off).mean(1, keepdim=True)
    evar = (DEPTH + 4) * U * var + 2 * em * em + 4 * U * em * off.abs().mean(1, keepdim=True)
    share = evar / (var + eps) + 4 * U
    assert bool((share < 0.5).all())
    rstd = (var + eps) ** -0.5
    w = 1.0 if weight is None else weight
    y = off * rstd * w
    ey = (eoff * (1 + share) + off.abs() * (share + 3 * U)) * rstd * abs(w)
    if bias is not None:
        y = y + bias
        ey = ey + U * (y.abs() + bias.abs())
    return y, ey + 2 * U * y.abs(), mean[:, 0], em[:, 0], rstd[:, 0], (rstd * share)[:, 0]


def layer_norm_backward(dy, x, mean, rstd, weight, residual):
    """{name: (value, its error)} of dx, dweight and dbias."""
    d, m = x.shape[1], x.shape[0]
    r = rstd[:, None]
    n = (x - mean[:, None]) * r
    g = dy if weight is None else dy * weight
    gn = g * n
    mg, mgn = g.mean(1, keepdim=True), gn.mean(1, keepdim=True)
    emg = (DEPTH + 2) * U * g.abs().mean(1, keepdim=True)
    emgn = (DEPTH + 8) * U * gn.abs().mean(1, keepdim=True)
    dx = r * (g - mg - n * mgn)
    size = g.abs() + mg.abs() + (n * mgn).abs()
    e = r * (emg + n.abs() * emgn + 8 * U * size)
    if residual is not None:
        dx = dx + residual
        e = e + 2 * U * (dx.abs() + residual.abs())
    return {"dx": (dx, e), "dweight": ((dy * n).sum(0), (m + 8) * U * (dy * n).abs().sum(0)),
            "dbias": (dy.sum(0), (m + 4) * U * dy.abs().sum(0))}


def philox(counter, key):
    """Philox4x32-10 of four arrays of 32-bit words in numpy's uint64."""
    mask, half = np.uint64(0xFFFFFFFF), np.uint64(32)
    c, (k0, k1) = list(counter), key
    for _ in range(10):
        p, q = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(q >> half) ^ c[1] ^ np.uint64(k0), q & mask, (p >> half) ^ c[3] ^ np.uint64(k1), p & mask]
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    return c


def draws(m, d, seed, offset):
    """The 16 bits of each element, as numbers [m, d]."""
    groups, low = (d + 7) // 8, 0xFFFFFFFF
    counter = [np.broadcast_to(np.arange(groups, dtype=np.uint64), (m, groups)),
               np.broadcast_to(np.arange(m, dtype=np.uint64)[:, None], (m, groups)),
               np.full((m, groups), offset & low, np.uint64), np.full((m, groups), offset >> 32, np.uint64)]
    words = np.stack(philox(counter, (seed & low, seed >> 32)), 2).astype(np.int64)
    return np.stack([words & 0xFFFF, words >> 16], 3).reshape(m, groups * 8)[:, :d]


def kept(p):
    return int(np.floor((1 - p) * 65536 + 0.5))
