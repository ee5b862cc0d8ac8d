"""CPU oracle of the attention operators (include/spec_attention.h).

TEST INFRASTRUCTURE, like the rest of ``oracle/``.  The definition, row by
row, in fp64: out = sum softmax(scale q.k) v over the visible keys, 0 (and a
log-sum-exp of -inf) where none is visible.  Beside each result the row's
rounding-free magnitudes are returned, from which the tests derive what an
f32-accumulating kernel may differ by.
"""
from __future__ import annotations

import math

import numpy as np


def ancestors(parents) -> np.ndarray:
    """bool [N][N]: node j is node i or one of its ancestors (parents[i] < i, -1 for the root)."""
    N = len(parents)
    out = np.zeros((N, N), dtype=bool)
    for i in range(N):
        a = i
        while a >= 0:
            out[i, a] = True
            a = int(parents[a])
    return out


def rows(q, k, v, visible, scale: float):
    """q [n][heads][D], k and v [m][kv_heads][D] fp64, visible bool [n][m].

    Returns out [n][heads][D], lse [n][heads], weight [n][heads][D] = sum
    softmax |v| and reach [n][heads] = max over the visible keys of
    scale * sum_d |q_d k_d| (0 without one).  Keys and values nobody sees take
    no part, whatever they hold."""
    n, heads, D = q.shape
    share = heads // k.shape[1]
    out = np.zeros((n, heads, D))
    weight = np.zeros((n, heads, D))
    lse = np.full((n, heads), -math.inf)
    reach = np.zeros((n, heads))
    for i in range(n):
        at = np.nonzero(visible[i])[0]
        if len(at) == 0:
            continue
        for h in range(heads):
            kk, vv = k[at, h // share], v[at, h // share]
            with np.errstate(invalid="ignore", over="ignore"):
                s = scale * (kk @ q[i, h])
                m = np.nan if np.isnan(s).any() else s.max()
                if m == -math.inf:
                    continue
                w = np.exp(s - m)
                total = w.sum()
                out[i, h] = (w[:, None] * vv).sum(0) / total
                weight[i, h] = (w[:, None] * np.abs(vv)).sum(0) / total
                lse[i, h] = m + np.log(total)
                reach[i, h] = scale * (np.abs(kk) @ np.abs(q[i, h])).max()
    return out, lse, weight, reach


def chain_mask(n: int, m: int) -> np.ndarray:
    """Causal, aligned at the end: query i of n sees key j of m iff j <= i + m - n."""
    return np.arange(m)[None, :] <= np.arange(n)[:, None] + (m - n)
