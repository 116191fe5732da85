"""Oracle: logit rows restricted by top-k, top-p and min-p, the sampler and the
verify on them, and the rotated append to a paged cache; fp64, one row at a time.

TEST INFRASTRUCTURE ONLY (see the package docstring for who may import it).

Readings (the rskf.cn survey, section 2.1, names top-p and temperature sampling
and gives no formulas):

* F1  the order: logits descending, equal logits by index; -inf and NaN logits
      are never kept.
* F2  one filter after the other: the first k; of those, a token is kept iff
      the share of the tokens before it is below p; of those, iff its
      probability is at least min_p times the largest.  The first is always
      kept.  0, 1 and 0 switch them off.
* F3  T = 0 keeps the first token alone.
* F4  a row without a logit above -inf keeps nothing; token 0 stands for it.
* F5  the verify is that of ``verify.verify_sample`` with the filtered p; a
      draft with p = 0 is rejected.
"""
from __future__ import annotations

from typing import NamedTuple

import numpy as np


class Row(NamedTuple):
    probs: np.ndarray     # [V]
    scale: float
    inv_sum: float
    max: float
    min_kept: float
    last: int
    n_kept: int


def filter_row(z, T: float, k: int = 0, p: float = 1.0, mp: float = 0.0) -> Row:
    z = np.asarray(z, dtype=np.float64)
    z = np.where(np.isnan(z), -np.inf, z)
    V = z.shape[0]
    T, p, mp = float(np.float32(T)), float(np.float32(p)), float(np.float32(mp))
    order = np.argsort(-z, kind="stable")
    order = order[z[order] > -np.inf]
    if order.size == 0:
        return Row(np.zeros(V), np.log2(np.e) / T if T else 0.0, 0.0, -np.inf, np.inf, -1, 0)
    m = z[order[0]]
    off = T > 0 and (k == 0 or k >= V) and p >= 1 and mp <= 0
    if T == 0:
        order = order[:1]
        w = np.ones(1)
    else:
        if k:
            order = order[:k]
        with np.errstate(invalid="ignore"):
            w = np.where(z[order] == m, 1.0, np.exp((z[order] - m) / T))
        if p < 1:
            before = np.concatenate(([0.0], np.cumsum(w)[:-1]))
            order, w = order[before < p * w.sum()], w[before < p * w.sum()]
        if mp > 0:
            order, w = order[w >= mp], w[w >= mp]
    q = np.zeros(V)
    q[order] = w / w.sum()
    return Row(q, np.log2(np.e) / T if T else 0.0, 1.0 / w.sum(), float(m),
               -np.inf if off else float(z[order[-1]]), V - 1 if off else int(order[-1]),
               V if off else int(order.size))


def draw(w: np.ndarray, u: float):
    """(token, distance): the inverse-CDF draw from masses w, and how far u's
    point lies from the drawn token's borders, as a share of the sum."""
    S = w.sum()
    if not S > 0:
        return 0, np.inf
    cum = np.cumsum(w)
    over = np.nonzero((cum > u * S) & (w > 0))[0]
    t = int(over[0]) if over.size else int(np.nonzero(w)[0][-1])
    edges = [abs(cum[t] - u * S)] + ([abs(cum[t] - w[t] - u * S)] if cum[t] - w[t] > 0 else [])
    return t, min(edges) / S


def verify_seq(rows, q, d, u, T):
    """(accepted, new token, p of the drafts, distance of the closest decision)
    of one sequence: rows [K+1] Row, q [K, V], d [K], u [K+1]."""
    K = len(d)
    p = np.array([rows[k].probs[d[k]] if 0 <= d[k] < len(rows[k].probs) else 0.0
                  for k in range(K)])
    near, a = np.inf, K
    for k in range(K):
        inside = 0 <= d[k] < len(rows[k].probs)
        if T == 0:
            ok = inside and d[k] == rows[k].last
        else:
            x = float(u[k]) * (q[k][d[k]] if inside else 0.0)
            ok = p[k] > 0 and x < p[k]
            if p[k] > 0:
                near = min(near, abs(x - p[k]) / p[k])
        if not ok:
            a = k
            break
    r = rows[a].probs
    if a < K and T > 0:
        res = np.maximum(0.0, r - q[a])
        r = res if res.sum() > 0 else r
    c, dist = draw(r, 0.0 if T == 0 else float(u[K]))
    return a, c, p, min(near, dist if T > 0 else np.inf)


def rotate(x, positions, inv_freq, interleaved: bool, scale: float = 1.0):
    """x [R, H, D] with its first 2 * len(inv_freq) elements rotated."""
    x = np.asarray(x, dtype=np.float64).copy()
    half = len(inv_freq)
    t = np.asarray(positions, np.float64)[:, None] * np.asarray(inv_freq, np.float64)
    c, s = np.cos(t)[:, None] * scale, np.sin(t)[:, None] * scale
    i0 = 2 * np.arange(half) if interleaved else np.arange(half)
    i1 = i0 + 1 if interleaved else i0 + half
    x0, x1 = x[..., i0].copy(), x[..., i1].copy()
    x[..., i0] = x0 * c - x1 * s
    x[..., i1] = x1 * c + x0 * s
    return x
