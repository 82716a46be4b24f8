"""CPU oracle of normed heads, attention weights and eviction -- TEST INFRASTRUCTURE ONLY.

Plain numpy float64 definitions: the RMS norm of a head with its gain and the rotary
positions, with their gradient; the attention weights of query rows, summed per cached
token and KV head; the choice and the move of the rows that an eviction keeps.  Shares
no code with the CUDA library.
"""
from __future__ import annotations

import numpy as np

from oracle import cache_ops as C


def norm_rope(x, gain, positions, freq, eps, layout):
    """x [tokens, heads, d]: R(p) (x / sqrt(mean x^2 + eps) * gain)."""
    n = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * gain
    return C.rope(n, positions, freq, 1.0, layout, False)


def norm_rope_backward(dy, x, gain, positions, freq, eps, layout):
    """(gradient of x, gradient of the gain) of sum(dy * norm_rope(x))."""
    d = x.shape[-1]
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    dn = C.rope(dy, positions, freq, 1.0, layout, True)
    u = dn * gain
    return r * u - x * r ** 3 * (u * x).sum(-1, keepdims=True) / d, (dn * x * r).sum((0, 1))


def probabilities(q, k, scale, first):
    """softmax(scale q k^T) of q [n, G, d] over k [m, d] rows, row i seeing keys 0 .. first + i: [n, G, m]; rows
    without a key are zeros."""
    n, m = q.shape[0], k.shape[0]
    s = np.einsum("igd,md->igm", q, k) * scale
    s = np.where(np.arange(m)[None, None, :] <= (first + np.arange(n))[:, None, None], s, -np.inf)
    top = s.max(-1, keepdims=True, initial=-np.inf)
    p = np.exp(s - np.where(np.isfinite(top), top, 0.0))
    total = p.sum(-1, keepdims=True)
    return np.divide(p, total, out=np.zeros_like(p), where=total > 0)


def keep_rows(weights, keep, sinks, recent):
    """Ascending rows that an eviction keeps of one sequence and KV head: weights [n].  The last `recent`, of the rest
    the first `sinks`, of the rest those of the largest weight (NaN below all numbers, ties to the lowest row), `keep` in all."""
    n = len(weights)
    if keep >= n:
        return np.arange(n)
    last = min(recent, keep)
    front = min(sinks, keep - last)
    middle = [(np.isnan(weights[i]), -np.nan_to_num(weights[i], nan=0.0, posinf=np.inf, neginf=-np.inf), i)
              for i in range(front, n - last)]
    chosen = sorted(i for _, _, i in sorted(middle)[:keep - last - front])
    return np.array(list(range(front)) + chosen + list(range(n - last, n)), dtype=np.int64)
