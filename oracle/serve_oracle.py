"""Plain fp64 oracle of the operators around the weight products (rotary
positions, quantised cache, attention over it, token scores), on the CPU.
Shares no code with the GPU library: NumPy on dense arrays, no pages, no tiles.
"""
from __future__ import annotations

import math

import numpy as np

TOP = {"e4m3": 448.0, "int8": 127.0}


def rope(x, positions, freqs, interleaved=False, inverse=False, table=None):
    """Rotation of the first 2 len(freqs) dims of x [T, H, D]; or, with table
    [P, r] (cosines, then sines), by its rows."""
    x = np.asarray(x, np.float64)
    if table is None:
        a = np.asarray(positions, np.float64)[:, None] * np.asarray(freqs, np.float64)[None]
        cos, sin = np.cos(a), np.sin(a)
    else:
        rows = np.asarray(table, np.float64)[np.asarray(positions)]
        cos, sin = np.split(rows, 2, axis=1)
    r = 2 * cos.shape[1]
    z = cos + 1j * (-sin if inverse else sin)
    y = x.copy()
    if interleaved:
        w = (x[..., 0:r:2] + 1j * x[..., 1:r:2]) * z[:, None]
        y[..., 0:r:2], y[..., 1:r:2] = w.real, w.imag
    else:
        w = (x[..., :r // 2] + 1j * x[..., r // 2:r]) * z[:, None]
        y[..., :r // 2], y[..., r // 2:r] = w.real, w.imag
    return y


def scale_of(x, fmt):
    """Scale [T, H] of heads x [T, H, D] (finite)."""
    amax = np.abs(np.asarray(x, np.float64)).max(-1)
    return np.where(amax >= 2.0 ** -100, amax / TOP[fmt], 0.0)


def half_step(y, fmt):
    """Half the distance of neighbouring codes at y (in units of the scale)."""
    y = np.abs(np.asarray(y, np.float64))
    if fmt == "int8":
        return np.full_like(y, 0.5)
    return 2.0 ** (np.floor(np.log2(np.maximum(y, 2.0 ** -6))) - 4)


def e4m3_values():
    """The 256 values of the format (4 exponent bits, bias 7, 3 mantissa bits;
    all ones is NaN, no infinities)."""
    out = np.empty(256)
    for b in range(256):
        e, m = (b >> 3) & 15, b & 7
        v = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        out[b] = (math.nan if (b & 127) == 127 else v) * (-1 if b & 128 else 1)
    return out


def attention(q, k, v, visible, scale):
    """q [n, Hq, D], k and v [L, H, D], visible [n, L]. Returns out, lse, the
    mean magnitude of values under the weights [n, Hq, D] and the largest
    sum_d |q_d k_d| |scale| over visible tokens [n, Hq] (for error bounds).
    Invisible tokens take no part, whatever they hold."""
    q, k, v = (np.asarray(a, np.float64) for a in (q, k, v))
    n, Hq, D = q.shape
    G = Hq // k.shape[1]
    out = np.zeros((n, Hq, D))
    mag = np.zeros((n, Hq, D))
    lse = np.full((n, Hq), -np.inf)
    big = np.zeros((n, Hq))
    for i in range(n):
        at = np.flatnonzero(visible[i])
        if len(at) == 0:
            continue
        for h in range(Hq):
            kk, vv = k[at, h // G], v[at, h // G]
            s = kk @ q[i, h] * scale
            m = s.max()
            p = np.exp(s - m)
            z = p.sum()
            out[i, h] = p @ vv / z
            mag[i, h] = p @ np.abs(vv) / z
            lse[i, h] = m + np.log(z)
            big[i, h] = (np.abs(kk) @ np.abs(q[i, h])).max() * abs(scale)
    return out, lse, mag, big


def tree_visible(length, n, rows=None):
    """[n, length]: causal, or by rows[i] = set of drafted tokens that i sees."""
    prefix = length - n
    see = np.zeros((n, length), bool)
    for i in range(n):
        for t in range(length):
            j = t - prefix
            see[i, t] = j < 0 or (j <= i if rows is None else j in rows[i])
    return see


def token_logprobs(x, ids, k):
    """Log probabilities of ids, entropy, top-k log probabilities and ids."""
    x = np.asarray(x, np.float64)
    m = x.max(-1, keepdims=True)
    with np.errstate(divide="ignore", invalid="ignore"):
        e = np.exp(x - m)
        z = e.sum(-1, keepdims=True)
        lp = x - m - np.log(z)
        p = e / z
        H = -np.where(p > 0, p * lp, 0.0).sum(-1)
    order = np.argsort(-x, axis=-1, kind="stable")[:, :k]
    rows = np.arange(len(x))
    return lp[rows, np.clip(ids, 0, x.shape[1] - 1)], H, np.take_along_axis(lp, order, 1), order
