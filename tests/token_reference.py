"""The token operators' formulas in 64 bits, and how far a result that holds
its sums and states in binary32 and rounds once may be from them.

U is half a step of binary32 at 1.  A sum over a row goes through at most
DEPTH additions on the way of any of its terms: 64 by one thread, 10 between
threads, and what makes the terms; so it is off by DEPTH * U of the sum of the
magnitudes.  Outputs are rounded by half a step of their type
(layer_reference.rounding)."""

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
