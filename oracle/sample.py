"""fp64 oracle of truncated sampling: min-p, top-k, top-p by row, and draws.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).

The pages name temperature and top-p, "applied identically to p and q before
the test" (pigeon guide, *When it breaks*); top-k and min-p are truncations of
the same kind.  Readings:

* min-p keeps p(x) >= min_p * max p, top-k every logit not below the k-th
  largest, top-p (on what those leave, renormalised) every logit not below the
  one where the descending cumulative mass first reaches top_p: a row is cut at
  one logit, ties included.
* A draw is the inverse CDF in id order over what is kept.
* T = 0: the largest logit's lowest id alone.  NaN counts as -inf; a logit of
  -inf is never kept; where a logit is +inf only those are, with equal weights.
"""
from __future__ import annotations

from dataclasses import dataclass

import numpy as np


@dataclass
class Kept:
    keep: np.ndarray    # bool [V]
    p: np.ndarray       # fp64 [V], 0 where not kept
    margin: float       # distance of the nucleus's mass from the next token's border, as a part of the total


def truncate(z, T: float, k: int = 0, top_p: float = 1.0, min_p: float = 0.0) -> Kept | None:
    """What a row keeps (None: no logit above -inf)."""
    z = np.array(z, dtype=np.float64)
    z[np.isnan(z)] = -np.inf
    M = z.max()
    if M == -np.inf:
        return None
    V = len(z)
    if T == 0:
        keep = np.zeros(V, bool)
        keep[int(np.flatnonzero(z == M)[0])] = True
        return Kept(keep, keep.astype(np.float64), np.inf)
    if M == np.inf:
        w = (z == np.inf).astype(np.float64)
        keep = w > 0
    else:
        with np.errstate(over="ignore", under="ignore"):
            w = np.exp((z - M) / T)
        keep = z > -np.inf
        if min_p > 0:
            keep &= z >= M + T * np.log(min_p)
    if 0 < k < V:
        keep &= z >= np.sort(z)[V - k]
    margin = np.inf
    if top_p < 1:
        vals, inv = np.unique(z[keep], return_inverse=True)  # ascending
        mass = np.zeros(len(vals))
        np.add.at(mass, inv, w[keep])
        down = np.cumsum(mass[::-1])  # descending
        target = top_p * down[-1]
        i = int(np.searchsorted(down, target))
        margin = np.abs(down - target).min() / down[-1]
        keep &= z >= vals[::-1][min(i, len(vals) - 1)]
    w = np.where(keep, w, 0.0)
    return Kept(keep, w / w.sum(), margin)


def draw(kept: Kept, u: float) -> tuple[int, float]:
    """(token, distance of u from the nearest border of the kept ids' cumulative mass)."""
    ids = np.flatnonzero(kept.keep)
    c = np.cumsum(kept.p[ids])
    x = min(max(float(u), 0.0), 1.0) * c[-1]
    i = int(np.searchsorted(c, x, side="right"))
    i = min(i, int(np.flatnonzero(kept.p[ids])[-1]))
    borders = np.concatenate([[0.0], c])
    inner = borders[1:-1]
    return int(ids[i]), float(np.abs(inner - x).min()) if len(inner) else np.inf
