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


def gate_errors(z, f, r, dtype):
    """Of f = 1 / (1 + E) and r = E f, relative to them, E = exp(-z) as a power of 2.

    E is off by its own step, 2 U, and by its exponent's rounding: z * log2(e) is off by half a step of itself,
    so E by |z| U, and by the constant's own share, 2^-25.2 of |z|, 0.4 |z| U; for binary32 rows both are made good to first
    order: 4 U in all.  Through 1 + E this reaches f by the share r = E / (1 + E) and r = E f by f.  To that come
    the sum's rounding, U, the reciprocal's step, 2 U, and r's product, U."""
    exponent = (4 * U if dtype == torch.float32 else (1.4 * z.abs() + 2) * U)
    return r * exponent + 3 * U, f * exponent + 4 * U


# Additions between parts of a sequence, on the way of any term.
PARTS = 40 * U


def places(offsets, m):
    """Row numbers of the sequences [batch, longest] and which of these places hold one, from the host's offsets."""
    begin = torch.tensor(offsets[:-1], dtype=torch.int64, device="cuda")
    length = torch.tensor(offsets[1:], dtype=torch.int64, device="cuda") - begin
    step = torch.arange(int(length.max()) if len(length) else 0, device="cuda")
    valid = step < length[:, None]
    return torch.where(valid, begin[:, None] + step, 0), valid


def lay(v, row, valid, other):
    return torch.where(valid[:, :, None], v.double()[row], other) if row.numel() else v.new_zeros((*row.shape, v.shape[1]), dtype=torch.float64)


def back(v, row, valid, m):
    out = torch.zeros((m, v.shape[2]), dtype=torch.float64, device="cuda")
    out[row[valid]] = v[valid]
    return out


def recurrence(gate, x, h0, offsets):
    """(h, its error, state, its error), row by row.

    A term that is t steps old has gone through t products with an f: each adds the error of that and a rounding.
    The magnitudes' own recurrence carries that along."""
    m, d = x.shape
    row, valid = places(offsets, m)
    gf, gr = gate_errors(*(lay(v, row, valid, 0.0) for v in (gate, torch.sigmoid(gate.double()), torch.sigmoid(-gate.double()))),
                         x.dtype)
    f, r = lay(torch.sigmoid(gate.double()), row, valid, 1.0), lay(torch.sigmoid(-gate.double()), row, valid, 0.0)
    xs = lay(x, row, valid, 0.0)
    now = torch.zeros(len(offsets) - 1, d, dtype=torch.float64, device="cuda")
    now = now if h0 is None else now + h0
    size, e = now.abs(), torch.zeros_like(now)
    h, eh = torch.zeros_like(f), torch.zeros_like(f)
    for t in range(row.shape[1]):
        on = valid[:, t, None]
        e = torch.where(on, f[:, t] * (e + (gf[:, t] + 2 * U) * size) + (gr[:, t] + 2 * U) * r[:, t] * xs[:, t].abs(), e)
        now = f[:, t] * now + r[:, t] * xs[:, t]
        size = f[:, t] * size + r[:, t] * xs[:, t].abs()
        h[:, t], eh[:, t] = now, e + PARTS * size
    return back(h, row, valid, m), back(eh, row, valid, m), now, e + PARTS * size


def recurrence_backward(dh, gate, x, h, h0, dstate, offsets):
    """{name: (value, its error)} of dgate, dx and dh0."""
    m, d = x.shape
    row, valid = places(offsets, m)
    gf, gr = gate_errors(*(lay(v, row, valid, 0.0) for v in (gate, torch.sigmoid(gate.double()), torch.sigmoid(-gate.double()))),
                         x.dtype)
    f, r = lay(torch.sigmoid(gate.double()), row, valid, 1.0), lay(torch.sigmoid(-gate.double()), row, valid, 0.0)
    xs, dhs, hs = (lay(v, row, valid, 0.0) for v in (x, dh, h))
    n = len(offsets) - 1
    start = torch.zeros(n, d, dtype=torch.float64, device="cuda")
    start = start if h0 is None else start + h0
    before = torch.cat([start[:, None], hs], 1)[:, :row.shape[1]]
    now = torch.zeros(n, d, dtype=torch.float64, device="cuda")
    now = now if dstate is None else now + dstate
    size, e = now.abs(), torch.zeros_like(now)
    g, eg = torch.zeros_like(f), torch.zeros_like(f)
    for t in reversed(range(row.shape[1])):
        on = valid[:, t, None]
        g[:, t] = now + dhs[:, t]
        size = size + dhs[:, t].abs()
        eg[:, t] = e + PARTS * size
        e = torch.where(on, f[:, t] * (e + (gf[:, t] + 2 * U) * size), e)
        now, size = f[:, t] * g[:, t], f[:, t] * size
    dx, edx = r * g, r * (eg + (gr + 2 * U) * g.abs())
    off = before - xs
    dgate = g * off * f * r
    edgate = f * r * off.abs() * (eg + (gf + gr + 6 * U) * g.abs())
    return {"dgate": (back(dgate, row, valid, m), back(edgate, row, valid, m)),
            "dx": (back(dx, row, valid, m), back(edx, row, valid, m)), "dh0": (now, e + PARTS * size)}
