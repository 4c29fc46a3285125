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


def pack4(w, group, rounded):
    """(codes, scales) of weights (out, in); ``rounded`` rounds an array to the scales' type."""
    w = np.asarray(w, dtype=np.float64)
    n, k = w.shape
    codes, scales = np.zeros((n, k)), np.zeros((n, -(-k // group)))
    for i in range(scales.shape[1]):
        part = w[:, i * group:(i + 1) * group]
        with np.errstate(invalid="ignore", divide="ignore"):
            s = rounded(np.abs(part).max(axis=1, initial=0.0) / 7)
            q = np.rint(part / s[:, None])
        usable = (s > 0) & np.isfinite(s)
        codes[:, i * group:(i + 1) * group] = np.where(usable[:, None], np.clip(q, -7, 7), 0.0)
        scales[:, i] = s
    return codes, scales


def values4(codes, scales, group):
    with np.errstate(invalid="ignore"):
        return codes * np.repeat(scales, group, axis=1)[:, :codes.shape[1]]
