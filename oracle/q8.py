"""Plain float64 oracle of the 8-bit latent cache and of the sampled tree verification
(test infrastructure; shares no code with the library).

The format (include/kdt.h): a cache row is 512 e4m3 codes, 16 power-of-two scale bytes (one
for each 32 codes, byte s for 2^(s-127), 255 for a group that reads as NaN) and 64 rope
values. e4m3 has 1 sign, 4 exponent (bias 7) and 3 mantissa bits; exponent 0 is subnormal
(mantissa/8 * 2^-6); the largest value is 448.
"""
from __future__ import annotations

import math

import numpy as np

GROUP = 32


def _code_values():
    v = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = (m / 8.0) * 2.0 ** -6 if e == 0 else (1.0 + m / 8.0) * 2.0 ** (e - 7)
        v[c] = -x if c & 0x80 else x
    v[0x7F] = v[0xFF] = np.nan
    return v


CODES = _code_values()


def dequantise(codes, scale):
    """codes uint8 [..., 512], scale uint8 [..., 16] -> float64 [..., 512]."""
    s = np.where(scale == 255, np.nan, np.exp2(scale.astype(np.float64) - 127.0))
    return CODES[codes] * np.repeat(s, GROUP, axis=-1)


def scale_exponent(top):
    """The least e in [-100, 100] with top <= 448 * 2^e (100 where there is none)."""
    e = np.full(top.shape, 100)
    for k in range(99, -101, -1):
        e = np.where(top <= 448.0 * 2.0 ** k, k, e)
    return e


def norm(x, gamma, eps):
    """RMS norm of float64 rows [..., 512]."""
    if gamma is None:
        return x
    return x / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps) * gamma


def rope(k, pos, base):
    """NeoX rotation of k [..., 64] at positions pos [...], float64."""
    half = k.shape[-1] // 2
    a = pos[..., None].astype(np.float64) * base ** (-np.arange(half, dtype=np.float64) / half)
    c, s = np.cos(a), np.sin(a)
    return np.concatenate([k[..., :half] * c - k[..., half:] * s, k[..., half:] * c + k[..., :half] * s], axis=-1)


def ancestors(parent):
    """bool [T,T]: node t is node i itself or an ancestor of it."""
    T = len(parent)
    see = np.zeros((T, T), dtype=bool)
    for i, p in enumerate(parent):
        if p >= 0:
            see[i] = see[p]
        see[i, i] = True
    return see


def attention(q, c, k_pe, prefix, see, scale):
    """One sequence: q [T,H,576], c [N,512], k_pe [N,64] float64 rows 0..prefix+T, see bool [T,T].
    Returns (out [T,H,512], lse [T,H]); a row that sees no key gets 0 and -inf. Hidden rows
    do not enter at all, whatever they hold."""
    T, H, _ = q.shape
    out, lse = np.zeros((T, H, 512)), np.full((T, H), -np.inf)
    for i in range(T):
        keys = np.concatenate([np.arange(prefix), prefix + np.flatnonzero(see[i])])
        if not len(keys):
            continue
        s = scale * (q[i, :, :512] @ c[keys].T + q[i, :, 512:] @ k_pe[keys].T)
        m = s.max(axis=-1, keepdims=True)
        p = np.exp(s - m)
        z = p.sum(axis=-1, keepdims=True)
        out[i] = (p @ c[keys]) / z
        lse[i] = (m + np.log(z))[:, 0]
    return out, lse


def sample_weights(logits, temperature):
    """Weights of one row, in units of 2^-44 of the largest (float64 integers)."""
    y = (logits.astype(np.float64) - np.max(logits)) / temperature
    return np.floor(np.exp(y) * 2.0 ** 44 + 0.5)


def tree_sample(parent, tok, logits, u_node, u_bonus, temperature):
    """One sequence: logits callable (node -> float64 row [V]). Returns (path, bonus, logp)."""
    T = len(parent)
    node, path, logp = 0, [0], []
    while True:
        row = logits(node)
        if not np.isfinite(np.max(row)) or np.isnan(row).any():
            return path, -1, logp + [0.0]
        w = sample_weights(row, temperature)
        lw = (row - np.max(row)) / temperature - math.log(w.sum() / 2.0 ** 44)
        left, step = w.copy(), None
        for c in range(node + 1, T):
            if parent[c] != node or not 0 <= tok[c] < len(w):
                continue
            if u_node[c] * left.sum() < left[tok[c]]:
                step = c
                break
            left[tok[c]] = 0.0
        if step is None:
            run = np.cumsum(left)
            bonus = int(np.searchsorted(run, float(u_bonus) * run[-1], side="right"))
            return path, bonus, logp + [lw[bonus]]
        logp.append(lw[tok[step]])
        path.append(step)
        node = step
