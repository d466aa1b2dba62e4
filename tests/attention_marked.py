"""Long attention inputs in which every tile of 128 keys counts: its share of some output element exceeds many times the bound on the kernels' error, so that a tile that is
lost, doubled or taken from another place shows.  (Over random values a tile's share shrinks with the
length while the bound grows.)  A tile's mark is a large value in a column of its own, or shared with
tiles far away; all else is small.

The plain 64-bit forms here are those of attention_reference, for chosen rows and keys of a sequence.
"""
from __future__ import annotations

import numpy as np

from attention_reference import BF16, scores

TILE = 128
NOISE, MARK = 0.1, 2.0
QUERY = 0.3  # of the queries over a long cache: keys weigh about alike


def tolerance(value, bound, half=BF16):
    return bound + half * (np.abs(value) + bound) + 1e-30


def tiles_of(n):
    return [slice(i, min(n, i + TILE)) for i in range(0, n, TILE)]


def mark_rows(rng, n, D, first=0, step=1, offset=0, size=MARK):
    """[n, D]: noise, and a mark for each tile of 128 rows in column first + (tile * step + offset) of the rest."""
    x = NOISE * rng.standard_normal((n, D))
    for i, t in enumerate(tiles_of(n)):
        x[t, first + (i * step + offset) % (D - first)] += size
    return x


# ------------------------------------------------------------------------------------- a long cache
def values_marked(rng, n, D):
    return mark_rows(rng, n, D, size=4.0)


def without_keys(q, k, v, seen, scale, keys):
    """The outputs of rows that lose ``keys`` (a slice), in 64 bits."""
    keep = seen.copy()
    keep[:, keys] = False
    z, _ = scores(q, k, scale)
    p = np.where(keep, np.exp(z - z.max(1, keepdims=True)), 0)
    return p @ v / p.sum(1, keepdims=True)
