"""Attention of the last tokens of a context under a sliding window with sinks, in plain numpy.

The token at position p sees token t <= p where t > p - window or t < sinks.  Everything in fp64,
from the definition: a mask, a softmax over what it leaves, a sum.
"""
from __future__ import annotations

import numpy as np


def seen(n: int, m: int, window: int | None, sinks: int) -> np.ndarray:
    """Truth [m, n]: which of n tokens the last m of them see (window None: all before them)."""
    p = np.arange(n - m, n)[:, None]
    t = np.arange(n)[None]
    near = t > p - window if window is not None else np.ones_like(t, bool)
    return (t <= p) & (near | (t < sinks))


def attention(q, k_rows, v_rows, scale, window=None, sinks=0):
    """q [m, Hq, d] of the last m of n tokens, k_rows / v_rows [h, n, d] -> [m, Hq, d]; rows of
    tokens that nothing sees may hold anything; a context without tokens gives zeros."""
    m, hq, d = q.shape
    h, n, _ = k_rows.shape
    if n == 0:
        return np.zeros((m, hq, d))
    mask = seen(n, m, window, sinks)
    live = mask.any(0)
    mask = mask[:, live]
    k, v = k_rows[:, live], v_rows[:, live]
    z = np.einsum("mhgd,hnd->mhgn", q.reshape(m, h, hq // h, d), k) * scale
    z = np.where(mask[:, None, None], z, -np.inf)
    p = np.exp(z - z.max(-1, keepdims=True))
    p /= p.sum(-1, keepdims=True)
    return np.einsum("mhgn,hnd->mhgd", p, v).reshape(m, hq, d)
