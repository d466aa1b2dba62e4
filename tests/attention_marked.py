"""Long attention inputs in which every tile of 128 keys, and every tile of rows of every head, counts: its
share of some output element exceeds many times the bound on the kernels' error, so that a tile that is
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


# ------------------------------------------------------------------------- gradients of a long prompt
def prompt_marked(rng, T, H, HK, D, heavy):
    """q, k, v, do [T, heads, D] of a prompt whose keys ``heavy`` weigh about alike in every row that sees
    them and about three times as much as all others together.

    k: tile j marked in a column (dq's shares); q, do: tile t of head g of its group marked (dk's and dv's);
    v and do: dP of tile j is +-4 by turns, so that dS keeps its sign within a tile."""
    G = H // HK
    q, do = (np.stack([mark_rows(rng, T, D, first=2, step=G, offset=h % G) for h in range(H)], 1) for _ in range(2))
    k = np.stack([mark_rows(rng, T, D, first=2) for _ in range(HK)], 1)
    v = NOISE * rng.standard_normal((T, HK, D))
    sign = np.where(np.arange(T) // TILE % 2 == 0, 1.0, -1.0)
    do[:, :, 0], v[:, :, 0] = 2.0, 2.0 * sign[:, None]
    q[:, :, 1], do[:, :, 1], k[:, :, 1], v[:, :, 1] = 4.0, 0.0, 0.0, 0.0
    scale = D ** -0.5
    k[list(heavy)] = NOISE * rng.standard_normal((len(heavy), HK, D))  # (their marks would hide those of other tiles)
    k[list(heavy), :, 1] = np.log(3.0 * T / len(heavy)) / (4.0 * scale)
    v[list(heavy), :, 0] = np.where(np.arange(len(heavy)) % 2 == 0, 2.0, -2.0)[:, None]
    return q, k, v, do, scale


def grad_pieces(q, k, v, scale, o, lse, do, seen, count):
    """The terms of attend_grad for some rows and keys of one head, and the errors of p and dS; ``count``:
    products in the kernels' sums."""
    D = q.shape[1]
    z, ez = scores(q, k, scale)
    with np.errstate(over="ignore"):
        p = np.where(seen, np.exp(np.where(seen, z - lse[:, None], 0)), 0)
    ep = p * (ez + np.abs(lse)[:, None] * 2.0 ** -22 + 2.0 ** -20)
    dp, delta = do @ v.T, (do * o).sum(1, keepdims=True)
    edp = (D + 2) * 2.0 ** -23 * (np.abs(do) @ np.abs(v).T + (np.abs(do) * np.abs(o)).sum(1, keepdims=True))
    ds = p * (dp - delta)
    eds = ep * np.abs(dp - delta) + p * edp + np.abs(ds) * (BF16 + 2.0 ** -21)
    return p, ep + p * BF16, ds, eds, (count + 4) * 2.0 ** -23


def rows_dq(q, k, v, scale, o, lse, do, rows):
    """dq of chosen rows of one head, (value, bound, [share of each tile of keys])."""
    n = max(rows) + 1
    seen = np.arange(n)[None] <= np.asarray(rows)[:, None]
    _, _, ds, eds, total = grad_pieces(q[rows], k[:n], v[:n], scale, o[rows], lse[rows], do[rows], seen, n)
    kk, s = k[:n], abs(scale)
    return scale * (ds @ kk), s * (eds @ np.abs(kk) + total * (np.abs(ds) @ np.abs(kk))), \
        [scale * (ds[:, t] @ kk[t]) for t in tiles_of(n)]


def keys_dkdv(q, k, v, scale, o, lse, do, keys):
    """dk and dv of chosen keys from one head, each (value, bound, [share of each tile of rows])."""
    T = q.shape[0]
    seen = np.asarray(keys)[None] <= np.arange(T)[:, None]
    p, ep, ds, eds, total = grad_pieces(q, k[keys], v[keys], scale, o, lse, do, seen, T)
    s = abs(scale)
    return {"dk": (scale * (ds.T @ q), s * (eds.T @ np.abs(q) + total * (np.abs(ds).T @ np.abs(q))),
                   [scale * (ds[t].T @ q[t]) for t in tiles_of(T)]),
            "dv": (p.T @ do, ep.T @ np.abs(do) + total * (p.T @ np.abs(do)), [p[t].T @ do[t] for t in tiles_of(T)])}


def weakest(value, bound, shares, seen):
    """The smallest, over rows and the tiles that they see, of a share's largest size in units of the tolerance:
    above 2, an output without that share is outside the tolerance whatever the kernel's own error."""
    tol = tolerance(value, bound)
    return min(float(np.max(np.abs(share[r]) / tol[r])) for r in range(value.shape[0]) for i, share in enumerate(shares) if seen(r, i))
