"""CPU fp64 definitions of the operators around a layer: embedding lookup, RMS norm with the residual's addition, its 8-bit
form, and Newton-Schulz steps.  Plain numpy from the formulas; shares nothing with the library."""
from __future__ import annotations

import numpy as np


def embed(index, table, scale, inner, column):
    out = np.zeros((len(index), table.shape[1], inner))
    for t, r in enumerate(index):
        if 0 <= r < table.shape[0]:
            out[t, :, column] = scale * table[r]
    return out


def embed_vjp(index, dout, rows, scale, column):
    """dtable, and for each row the sum of the magnitudes that were added and their number."""
    d = np.zeros((rows, dout.shape[1]))
    size, count = np.zeros_like(d), np.zeros(rows)
    keep = (index >= 0) & (index < rows)
    np.add.at(d, index[keep], dout[keep, :, column])
    np.add.at(size, index[keep], np.abs(dout[keep, :, column]))
    np.add.at(count, index[keep], 1)
    return scale * d, abs(scale) * size, count


def rms_norm(h, gamma, eps):
    """y and rstd of h [N][C][inner]."""
    n = h.shape[0]
    rstd = (np.mean(h.reshape(n, -1) ** 2, axis=1) + eps) ** -0.5 if n else np.zeros(0)
    return h * rstd[:, None, None] * gamma[None, :, None], rstd


def rms_norm_vjp(h, gamma, eps, dy, dh=None):
    """dx, dgamma of <dy, rms_norm(h)> + <dh, h>."""
    _, rstd = rms_norm(h, gamma, eps)
    u = h * rstd[:, None, None]
    t = dy * gamma[None, :, None]
    dx = rstd[:, None, None] * (t - u * np.mean(t * u, axis=(1, 2), keepdims=True))
    return dx if dh is None else dx + dh, np.sum(dy * u, axis=(0, 2))


def scales(y, group):
    """Scales of y [N][L] for groups of `group` values (0: a row)."""
    n, width = y.shape
    group = group or width
    return np.stack([np.abs(y[:, i:i + group]).max(1) for i in range(0, width, group)], 1) / 448.0


def e4m3_step(v):
    """Distance of e4m3 values about |v| <= 448: 3 bits after the first, the smallest 2^-9."""
    e = np.floor(np.log2(np.maximum(np.abs(v), 2.0 ** -6)))
    return 2.0 ** (e - 3)


def newton_schulz(g, steps, coefficients, eps):
    """The steps' results X_0 .. X_steps, on the smaller side."""
    a, b, c = coefficients
    x = np.asarray(g, np.float64)
    x = x / (np.linalg.norm(x) + eps)
    tall = x.shape[0] > x.shape[1]
    if tall:
        x = x.T
    xs = [x]
    for _ in range(steps):
        p = x @ x.T
        x = a * x + (b * p + c * p @ p) @ x
        xs.append(x)
    return [v.T for v in xs] if tall else xs
