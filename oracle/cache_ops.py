"""Plain fp64 forms (numpy) of the operators on caches whose slots are not one
token after the other: drafted trees, accumulated key weights, eviction. Loops
over rows and heads; shares no code with the CUDA path."""
from __future__ import annotations

import numpy as np


def tree_visible(parents):
    """[n, n] truth values: row i sees its ancestors and itself. parents[i] < i, -1 for a root."""
    n = len(parents)
    out = np.zeros((n, n), bool)
    for i in range(n):
        j = i
        while j >= 0:
            out[i, j] = True
            j = parents[j]
    return out


def mask_words(visible, words=None):
    """The truth values as int32 words, bit j % 32 of word j // 32 for row j."""
    n = visible.shape[1]
    words = max(1, -(-n // 32)) if words is None else words
    out = np.zeros((visible.shape[0], words), np.uint32)
    for j in range(min(n, 32 * words)):
        out[:, j // 32] |= visible[:, j].astype(np.uint32) << np.uint32(j % 32)
    return out.view(np.int32)


def weigh(q, K, pos, where, keep, scale, cap=0.0, slope=0.0):
    """Softmax weights of keys K [n, d] at positions `where` for one query at position pos;
    keep [n] marks the visible ones, the others weigh 0."""
    p = np.zeros(K.shape[0])
    if not np.any(keep):
        return p
    s = K[keep] @ q * scale
    if cap > 0:
        s = cap * np.tanh(s / cap)
    s = s - slope * np.abs(pos - where[keep])
    e = np.exp(s - s.max())
    p[keep] = e / e.sum()
    return p


def attend(q, K, V, pos, where, keep, scale, cap=0.0, slope=0.0):
    """(o, m): the output of one query and sum p |v|, what relative errors of the weights act on."""
    p = weigh(q, K, pos, where, keep, scale, cap, slope)
    return p[keep] @ V[keep], p[keep] @ np.abs(V[keep])


def evict(weights, keep, first, recent):
    """Ascending slots that stay of n = len(weights) filled ones."""
    n = len(weights)
    if n <= keep:
        return list(range(n))
    middle = sorted(range(first, n - recent), key=lambda i: (np.isnan(weights[i]), -weights[i], i))
    return sorted(list(range(first)) + middle[:keep - first - recent] + list(range(n - recent, n)))
