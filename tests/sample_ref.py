"""float64 reference of the rules that cut logits, and of the draw, on the CPU."""

from __future__ import annotations

import numpy as np


def kept(x, T, k=None, p=None, m=None):
    """One row of float64 logits (NaN: as -inf): the ids that the rules leave, ascending, and their weights."""
    x = np.where(np.isnan(x), -np.inf, x)
    order = np.lexsort((np.arange(x.size), -x))
    order = order[x[order] > -np.inf]
    if not order.size:
        return order, np.zeros(0)
    top = x[order[0]]
    with np.errstate(invalid="ignore", over="ignore"):
        w = np.where(x[order] == top, 1.0, np.exp((x[order] - top) / np.float64(T)))
    stay = np.ones(order.size, dtype=bool)
    if k is not None and 0 < k < x.size:
        stay[k:] = False
    if p is not None and p < 1:
        mass = np.cumsum(np.where(stay, w, 0.0))
        stay[1:] &= mass[:-1] < p * mass[-1]
    if m is not None and m > 0:
        stay &= w >= min(m, 1.0)
    ids, w = order[stay], w[stay]
    by = np.argsort(ids)
    return ids[by], w[by]


def draw(ids, w, u):
    """The token of uniform u, and its log-probability."""
    if not ids.size:
        return -1, -np.inf
    upto = np.cumsum(w)
    u = min(max(float(u), 0.0), 1.0 - 2.0 ** -24) if u == u else 0.0
    at = int(np.searchsorted(upto, u * upto[-1], side="right"))
    while at >= ids.size or w[at] == 0:
        at -= 1
    return int(ids[at]), float(np.log(w[at] / upto[-1]))


def greedy(x):
    x = np.where(np.isnan(x), -np.inf, x)
    return (int(np.argmax(x)), 0.0) if x.max() > -np.inf else (-1, -np.inf)
