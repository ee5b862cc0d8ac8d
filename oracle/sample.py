"""CPU oracle of filtered sampling (include/spec_sample.h).

TEST INFRASTRUCTURE, like the rest of ``oracle/``.  One row at a time, in fp64,
from the definition; beside the result, how far the nearest decision was from
its border, in units of the mass (a draw or a nucleus) or of the weight (min-p).
"""
from __future__ import annotations

import math

import numpy as np


def row(z, u, T: float, top_k: int = 0, top_p: float = 1.0, min_p: float = 0.0):
    """z [V] f32 values, u in [0, 1) or None.  Returns (token or None, kept bool [V], margin)."""
    z = np.asarray(z, dtype=np.float64)
    m = z.max()
    kept = np.zeros(len(z), dtype=bool)
    if T == 0:
        kept[int(np.argmax(z))] = True
        return int(np.argmax(z)), kept, math.inf
    T = min(max(T, 2.0 ** -100), 2.0 ** 100)
    with np.errstate(over="ignore", under="ignore"):
        w = np.exp((z - m) / T)
    order = np.argsort(-z, kind="stable")
    order = order[z[order] > -math.inf]
    margin = math.inf
    n = len(order)
    if top_k > 0:
        n = min(n, top_k)
    if top_p < 1:
        mass = np.cumsum(w[order[:n]])
        before = mass - w[order[:n]]
        inside = before < top_p * mass[-1]
        inside[0] = True
        margin = min(margin, np.abs(before[1:] / mass[-1] - top_p).min(initial=math.inf))
        n = int(inside.sum())
    order = order[:n]
    if min_p > 0:
        limit = min(min_p, 1.0)
        margin = min(margin, np.abs(w[order] / limit - 1)[w[order] != limit].min(initial=math.inf))
        order = order[w[order] >= limit]
    kept[order] = True
    if u is None:
        return None, kept, margin
    c = np.cumsum(np.where(kept, w, 0.0))
    over = np.nonzero(c > min(max(u, 0.0), 1.0) * c[-1])[0]
    token = int(over[0]) if len(over) else int(np.nonzero(kept & (w > 0))[0][-1])
    margin = min(margin, float(np.abs(c / c[-1] - u)[kept & (w > 0)].min()) if 0 < u < 1 else math.inf)
    return token, kept, margin


def filtered(z, kept, T: float):
    """The filtered logits, in f32."""
    z = np.asarray(z, dtype=np.float32)
    least, away = float(np.finfo(np.float32).min), 512.0 * (T if T > 0 else 1.0)
    top = float(z.max())
    gone = np.float32(max(top - away, least))
    if top - float(gone) < 0.75 * away and gone > least:  # f32 is too coarse here: rounded away from the largest
        gone = max(np.nextafter(gone, np.float32(least)), np.float32(least))
    return np.where(kept, z, gone)
