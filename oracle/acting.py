"""Float64 definitions of what acting with the centre network takes: drawing an index from logits."""

import math

import numpy as np


def keep(x, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """(weights with those not kept at 0, or None for a row without an answer): one row of logits, one element at
    a time over the order."""
    x = np.asarray(x, dtype=np.float64)
    n = x.size
    if np.isnan(x).any() or x.max() == -math.inf:
        return None
    if temperature <= 0:
        top_k, temperature = 1, 1.0
    top = x.max()
    with np.errstate(invalid="ignore", over="ignore", under="ignore"):
        w = np.where(x == top, 1.0, np.exp((x - top) / temperature))
    order = sorted(range(n), key=lambda i: (-x[i], i))
    if 0 < top_k < n:
        order = order[:top_k]
    if top_p < 1:
        bound, before, cut = top_p * math.fsum(w[i] for i in order), 0.0, []
        for i in order:
            if cut and not before < bound:
                break
            cut.append(i)
            before += w[i]
        order = cut
    if min_p > 0:
        order = [i for i in order if w[i] >= min(min_p, 1.0)]
    kept = np.zeros(n)
    kept[order] = w[order]
    return kept


def sample(x, u, **filters):
    """(index, log of the share it has) of one row."""
    if any(math.isnan(v) for v in [u, *filters.values()]):
        return -1, math.nan
    w = keep(x, **filters)
    if w is None:
        return -1, math.nan
    c = np.cumsum(w)
    last = int(np.flatnonzero(w)[-1])
    i = min(int(np.searchsorted(c, max(u, 0.0) * c[-1], side="right")), last)
    return i, math.log(w[i] / c[-1])
