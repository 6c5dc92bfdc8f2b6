"""Oracle of the sampling calls: which tokens a row's filters keep, their
probabilities, and the token that a given number draws.

The definition in long doubles over a full sort of the row, with the distance of
every comparison from its border: where a compared mass lies closer to its
border than a caller's arithmetic can tell, either outcome is right.
"""
from __future__ import annotations

import numpy as np


def sample_filter(x, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """One row x [V] -> (w [V]: weights relative to the largest, 0 where not kept;
    margin: the least distance of a top-p comparison from its border, relative to
    the mass).  None for a row without a distribution."""
    x = np.asarray(x, dtype=np.longdouble)
    if np.any(np.isnan(x)) or np.max(x) in (np.inf, -np.inf) or np.isnan(top_p) or np.isnan(min_p) \
            or not 0 <= temperature < np.inf:
        return None
    if temperature == 0:
        temperature, top_k = 1.0, 1
    order = np.lexsort((np.arange(len(x)), -x))  # logit down, index up
    z = (x[order] - x[order[0]]) / np.longdouble(temperature)
    w = np.exp(z)
    keep = np.isfinite(x[order])
    if top_k > 0:
        keep &= np.arange(len(x)) < top_k
    if min_p > 0:  # in logarithms: exp(z) of a tiny z rounds to 1
        keep &= z >= np.log(min(np.longdouble(min_p), np.longdouble(1)))
    w = np.where(keep, w, 0)
    margin = 1.0
    if top_p < 1:
        total = w.sum()
        before = np.concatenate([[0], np.cumsum(w)[:-1]])
        keep &= before < np.longdouble(top_p) * total
        keep[0] = True
        off = np.abs(before[1:] - np.longdouble(top_p) * total)[w[1:] > 0] / total
        margin = float(off.min()) if len(off) else 1.0
        w = np.where(keep, w, 0)
    out = np.zeros(len(x), dtype=np.longdouble)
    out[order] = w
    return out, margin


def sample_token(w, u):
    """(token, margin): the least i whose cumulative w exceeds u sum(w), and the
    distance of u sum(w) from the nearest border, relative to the sum."""
    grown = np.cumsum(w)
    target = np.longdouble(min(max(float(u), 0.0), 1 - 2.0 ** -24)) * grown[-1]
    token = int(np.argmax(grown > target))
    borders = grown[np.asarray(w) > 0]
    return token, float(np.min(np.abs(borders - target)) / grown[-1])
