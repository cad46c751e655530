"""Plain fp64 forms (numpy) of the attention operators beside the Llama2 path:
head norms, half-split / partial / scaled rotation, and attention with capped
or biased scores, documents, two-way prefixes. Loops over rows and heads;
shares no code with the CUDA path."""
from __future__ import annotations

import math

import numpy as np


def rotation_table(n_pos, rotary_dim, theta=10000.0, kind="plain", factor=1.0, low_turns=1.0,
                   high_turns=32.0, original_len=4096, magnitude=1.0):
    """[n_pos, rotary_dim / 2, 2] of magnitude * (cos, sin)(position * f_j)."""
    out = np.empty((n_pos, rotary_dim // 2, 2))
    for j in range(rotary_dim // 2):
        f = theta ** (-2.0 * j / rotary_dim)
        if kind == "linear":
            f = f / factor
        elif kind == "bands":
            turns = original_len * f / (2 * math.pi)
            g = min(1.0, max(0.0, (turns - low_turns) / (high_turns - low_turns)))
            f = f * g + f / factor * (1 - g)
        a = np.arange(n_pos) * f
        out[:, j, 0], out[:, j, 1] = magnitude * np.cos(a), magnitude * np.sin(a)
    return out


def head_norm(x, gain, eps):
    """x [..., d] over its own d values."""
    return x / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps) * gain


def rotate(x, cs, half):
    """x [..., d]; cs [r / 2, 2] of the position; the first r values turn."""
    y = x.copy()
    n = cs.shape[0]
    for j in range(n):
        i0, i1 = (j, j + n) if half else (2 * j, 2 * j + 1)
        y[..., i0] = x[..., i0] * cs[j, 0] - x[..., i1] * cs[j, 1]
        y[..., i1] = x[..., i0] * cs[j, 1] + x[..., i1] * cs[j, 0]
    return y


def attend_row(q, K, V, pos, keep, scale, cap=0.0, slope=0.0):
    """One query q [d] at position pos over keys K, V [n, d] at positions 0..n-1;
    keep [n] marks the visible ones. Returns (o, m): o the output, m = sum p |v|
    (what relative errors of the weights act on). No visible key: zeros."""
    if not np.any(keep):
        return np.zeros(V.shape[1]), np.zeros(V.shape[1])
    s = K[keep] @ q * scale
    if cap > 0:
        s = cap * np.tanh(s / cap)
    s = s - slope * np.abs(pos - np.arange(K.shape[0])[keep])
    p = np.exp(s - s.max())
    p = p / p.sum()
    return p @ V[keep], p @ np.abs(V[keep])


def attend_documents(q, k, v, cu, prefix, scale, cap=0.0, slopes=None, rows=None):
    """q [n, n_q, d], k, v [n, n_kv, d]; documents cu; prefix [B] or None. Returns
    (out, mass) [n, n_q, d]; rows of no document (or not in `rows`) are NaN."""
    n, nq, d = q.shape
    G = nq // k.shape[1]
    out, mass = np.full((n, nq, d), np.nan), np.full((n, nq, d), np.nan)
    for b in range(len(cu) - 1):
        lo, hi = int(cu[b]), int(cu[b + 1])
        pre = 0 if prefix is None else int(prefix[b])
        j = np.arange(hi - lo)
        for r in range(lo, hi):
            if rows is not None and r not in rows:
                continue
            keep = (j <= r - lo) | (j < pre)
            for h in range(nq):
                out[r, h], mass[r, h] = attend_row(q[r, h], k[lo:hi, h // G], v[lo:hi, h // G], r - lo,
                                                   keep, scale, cap, 0.0 if slopes is None else slopes[h])
    return out, mass
