"""CPU fp64 definitions of the node-update operators: group norm with an activation, attention to another
set of states, dropout from a counter-based generator.

Plain numpy, graph by graph and head by head, from the formulas; shares nothing with the library.
Where a test needs an elementwise error bound for 16-bit operands, the functions also return the
first-order magnitude that a relative rounding of the probabilities and of the score gradients is
multiplied with.
"""
from __future__ import annotations

import numpy as np


def sigmoid(z):
    return 0.5 * (1 + np.tanh(0.5 * z))


def act(z, silu):
    return z * sigmoid(z) if silu else z


def act_grad(z, silu):
    if not silu:
        return np.ones_like(z)
    s = sigmoid(z)
    return s * (1 + z * (1 - s))


def group_norm(x, gamma, beta, offsets, groups, silu, eps):
    """y [N][C], mean [B][G], rstd [B][G]."""
    x = np.asarray(x, np.float64)
    c = x.shape[1]
    per = c // groups
    y = np.zeros_like(x)
    b = len(offsets) - 1
    mean, rstd = np.zeros((b, groups)), np.full((b, groups), eps ** -0.5 if eps > 0 else np.inf)
    for i in range(b):
        for g in range(groups):
            part = x[offsets[i]:offsets[i + 1], g * per:(g + 1) * per]
            if part.size == 0:
                continue
            m = part.mean()
            r = (((part - m) ** 2).mean() + eps) ** -0.5
            mean[i, g], rstd[i, g] = m, r
            z = (part - m) * r * gamma[g * per:(g + 1) * per] + beta[g * per:(g + 1) * per]
            y[offsets[i]:offsets[i + 1], g * per:(g + 1) * per] = act(z, silu)
    return y, mean, rstd


def group_norm_vjp(x, gamma, beta, offsets, groups, silu, eps, dy):
    """dx, dgamma, dbeta of <dy, group_norm(x)>."""
    x, dy = np.asarray(x, np.float64), np.asarray(dy, np.float64)
    _, mean, rstd = group_norm(x, gamma, beta, offsets, groups, silu, eps)
    per = x.shape[1] // groups
    dx, dg, db = np.zeros_like(x), np.zeros(x.shape[1]), np.zeros(x.shape[1])
    for i in range(len(offsets) - 1):
        for g in range(groups):
            at = np.s_[offsets[i]:offsets[i + 1], g * per:(g + 1) * per]
            ch = slice(g * per, (g + 1) * per)
            if x[at].size == 0:
                continue
            xh = (x[at] - mean[i, g]) * rstd[i, g]
            dz = dy[at] * act_grad(xh * gamma[ch] + beta[ch], silu)
            dg[ch] += (dz * xh).sum(0)
            db[ch] += dz.sum(0)
            t = dz * gamma[ch]
            dx[at] = rstd[i, g] * (t - t.mean() - xh * (t * xh).mean())
    return dx, dg, db


def _kept(i, k_offsets, keep):
    j = np.arange(k_offsets[i], k_offsets[i + 1])
    return j if keep is None else j[np.asarray(keep)[j] != 0]


def attention(q, k, v, q_offsets, k_offsets, scale, keep=None):
    """out [Tq][Hq][D], lse [Tq][Hq], and sum_j P_ij |v_j| like out."""
    q, k, v = (np.asarray(t, np.float64) for t in (q, k, v))
    hq, group = q.shape[1], q.shape[1] // k.shape[1]
    out, mag = np.zeros_like(q), np.zeros_like(q)
    lse = np.full(q.shape[:2], -np.inf)
    for i in range(len(q_offsets) - 1):
        rows, j = slice(q_offsets[i], q_offsets[i + 1]), _kept(i, k_offsets, keep)
        if j.size == 0:
            continue
        for h in range(hq):
            s = scale * q[rows, h] @ k[j, h // group].T
            top = s.max(1, keepdims=True)
            p = np.exp(s - top)
            total = p.sum(1, keepdims=True)
            lse[rows, h] = (top + np.log(total))[:, 0]
            p /= total
            out[rows, h] = p @ v[j, h // group]
            mag[rows, h] = p @ np.abs(v[j, h // group])
    return out, lse, mag


def attention_vjp(q, k, v, q_offsets, k_offsets, scale, d_out, keep=None, unit=0.0):
    """(dq, dk, dv) of <d_out, attention>, and for each the elementwise first-order bound of its error when P, dS and the
    results are rounded to relative `unit` and delta = d_out . out is formed from the rounded out."""
    q, k, v, d_out = (np.asarray(t, np.float64) for t in (q, k, v, d_out))
    hq, group = q.shape[1], q.shape[1] // k.shape[1]
    out, _, mag = attention(q, k, v, q_offsets, k_offsets, scale, keep)
    g = [np.zeros_like(t) for t in (q, k, v)]
    e = [np.zeros_like(t) for t in (q, k, v)]
    for i in range(len(q_offsets) - 1):
        rows, j = slice(q_offsets[i], q_offsets[i + 1]), _kept(i, k_offsets, keep)
        if j.size == 0 or q_offsets[i] == q_offsets[i + 1]:
            continue
        for h in range(hq):
            kk, vv, qq, do = k[j, h // group], v[j, h // group], q[rows, h], d_out[rows, h]
            s = scale * qq @ kk.T
            p = np.exp(s - s.max(1, keepdims=True))
            p /= p.sum(1, keepdims=True)
            ds = p * (do @ vv.T - (do * out[rows, h]).sum(1, keepdims=True)) * scale
            g[0][rows, h] = ds @ kk
            g[1][j, h // group] += ds.T @ qq
            g[2][j, h // group] += p.T @ do
            off = (np.abs(do) * (np.abs(out[rows, h]) + 2 * mag[rows, h])).sum(1, keepdims=True)
            de = unit * (np.abs(ds) + scale * p * off)
            e[0][rows, h] += de @ np.abs(kk)
            e[1][j, h // group] += de.T @ np.abs(qq)
            e[2][j, h // group] += unit * p.T @ np.abs(do)
    return g, [x + unit * np.abs(y) for x, y in zip(e, g)]


def philox(counter, seed):
    """Four 32-bit words of Philox4x32-10 for a 64-bit counter and a 64-bit key, in Python integers."""
    c = [counter & 0xFFFFFFFF, (counter >> 32) & 0xFFFFFFFF, 0, 0]
    k = [seed & 0xFFFFFFFF, (seed >> 32) & 0xFFFFFFFF]
    return philox_words(c, k)


def philox_words(c, k):
    """Philox4x32-10 of a full counter (4 words) and key (2 words)."""
    c, k = list(c), list(k)
    for _ in range(10):
        a, b = 0xD2511F53 * c[0], 0xCD9E8D57 * c[2]
        c = [(b >> 32) ^ c[1] ^ k[0], b & 0xFFFFFFFF, (a >> 32) ^ c[3] ^ k[1], a & 0xFFFFFFFF]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return c


def keep_mask(draws, p, seed, offset):
    """Booleans [draws] and the scale of kept values."""
    limit = int(np.floor(p * 65536 + 0.5))
    halves = []
    for block in range(-(-draws // 8)):
        for w in philox((offset + block) & 0xFFFFFFFFFFFFFFFF, seed):
            halves += [w & 0xFFFF, w >> 16]
    return np.array(halves[:draws], dtype=np.int64) >= limit, 65536 / (65536 - limit) if limit < 65536 else 0.0
