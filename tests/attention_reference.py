"""Plain 64-bit forms of the norm and rotation of queries and keys and of softmax attention (numpy),
each with a bound on the kernels' error computed alongside.

The bounds count what the kernels do: a rounding to FP32 is 2^-24 relative (2^-23 is counted for a
sum on the tensor cores, which may cut instead of round), exp2, log2, rsqrt and reciprocal 2^-22 at
most each, sine and cosine 2^-22 absolute, a rounding to BF16 2^-8.  Hence
    score        e_z = (D + 8) 2^-23 scale sum|q k| + |z| 2^-22      (absolute, also of z - lse)
    probability  p (e_z + 2^-21), rounded to BF16 as an operand: p 2^-8 more
and every sum of n products adds n 2^-23 of the sum of their absolute values.
"""
from __future__ import annotations

import numpy as np

BF16 = 2.0 ** -8
HALF_STEP = {"bf16": 2.0 ** -8, "fp32": 2.0 ** -24}


# ------------------------------------------------------------------------- norm and rotation
def rotation(positions, inv_freq):
    """cos, sin [tokens, 1, R/2] of the exact products, and their absolute error."""
    a = np.asarray(positions, dtype=np.float64)[:, None, None] * np.asarray(inv_freq, dtype=np.float64)
    return np.cos(a), np.sin(a), 2.0 ** -21 + np.abs(a) * 2.0 ** -51


def halves(R, interleaved):
    return (slice(0, R, 2), slice(1, R, 2)) if interleaved else (slice(0, R // 2), slice(R // 2, R))


def rotate(y, ey, cs, R, interleaved, back=False):
    """(rotated y, its error) for y [tokens, heads, D] with error ey."""
    out, e = y.copy(), ey.copy()
    if R:
        c, s, d = cs
        s = -s if back else s
        lo, hi = halves(R, interleaved)
        a, b, ea, eb = y[..., lo], y[..., hi], ey[..., lo], ey[..., hi]
        out[..., lo], out[..., hi] = a * c - b * s, a * s + b * c
        both = (np.abs(a) + np.abs(b)) * (d + 2.0 ** -22)
        e[..., lo] = ea * np.abs(c) + eb * np.abs(s) + both
        e[..., hi] = ea * np.abs(s) + eb * np.abs(c) + both
    return out, e


def norm_rope(x, w, eps, positions, inv_freq, interleaved):
    x = np.asarray(x, dtype=np.float64)
    D, R = x.shape[-1], 2 * len(inv_freq)
    w = np.ones(D) if w is None else np.asarray(w, dtype=np.float64)
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w
    ey = np.abs(y) * (0.5 * D * 2.0 ** -24 + 2.0 ** -21)
    return rotate(y, ey, rotation(positions, inv_freq), R, interleaved)


def norm_rope_grad(x, w, eps, dout, positions, inv_freq, interleaved):
    """dict name -> (value, bound): dx and the sum dweight."""
    x, dout = np.asarray(x, dtype=np.float64), np.asarray(dout, dtype=np.float64)
    D, R = x.shape[-1], 2 * len(inv_freq)
    w = np.ones(D) if w is None else np.asarray(w, dtype=np.float64)
    g, eg = rotate(dout, np.zeros_like(dout), rotation(positions, inv_freq), R, interleaved, back=True)
    rstd = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    n, wg, ewg = x * rstd, w * g, np.abs(w) * (eg + 2.0 ** -24 * np.abs(g))
    m = (wg * n).mean(-1, keepdims=True)
    dx = rstd * (wg - n * m)
    e = 0.5 * D * 2.0 ** -24 + 2.0 ** -21  # relative error of rstd and n
    em = (np.abs(wg * n) * (D * 2.0 ** -24 + 2 * e) + ewg * np.abs(n)).mean(-1, keepdims=True)
    edx = rstd * (np.abs(wg) * e + ewg + np.abs(n) * em + np.abs(n * m) * 3 * e
                  + 2.0 ** -22 * (np.abs(wg) + np.abs(n * m)))
    count = x.shape[0] * x.shape[1]
    size = np.abs(g * n).sum((0, 1))
    edw = size * (e + (count + 2) * 2.0 ** -24) + (eg * np.abs(n)).sum((0, 1))
    return {"dx": (dx, edx), "dw": ((g * n).sum((0, 1)), edw)}


# ------------------------------------------------------------------------------- attention
def scores(q, k, scale):
    """z = scale q k^T [rows, keys] and its absolute error."""
    z = scale * (q @ k.T)
    return z, (q.shape[1] + 8) * 2.0 ** -23 * abs(scale) * (np.abs(q) @ np.abs(k).T) + np.abs(z) * 2.0 ** -22


def attend(q, k, v, seen, scale):
    """One head's rows: (o, lse, bound of o, bound of lse); a row that sees nothing gives 0, -inf."""
    q, k, v = (np.asarray(t, dtype=np.float64) for t in (q, k, v))
    rows, n = q.shape[0], max(1, k.shape[0])
    o, lse = np.zeros((rows, v.shape[1])), np.full(rows, -np.inf)
    eo, el = np.zeros_like(o), np.zeros(rows)
    if k.shape[0] == 0:
        return o, lse, eo, el
    z, ez = scores(q, k, scale)
    z, ez = np.where(seen, z, -np.inf), np.where(seen, ez, 0)
    top = z.max(1, keepdims=True)
    live = np.isfinite(top[:, 0])
    with np.errstate(invalid="ignore"):
        p = np.where(seen & live[:, None], np.exp(z - np.where(np.isfinite(top), top, 0)), 0)
    total = p.sum(1, keepdims=True)
    p = p / np.where(total > 0, total, 1)
    worst = (p * ez).sum(1) + n * 2.0 ** -23 + 2.0 ** -20
    lse[live] = top[live, 0] + np.log(total[live, 0])
    el[live] = (worst + np.abs(lse, where=live, out=np.zeros(rows)) * 2.0 ** -22 + 2.0 ** -20)[live]
    # masked values reach nothing, whatever they are
    vv = np.where(np.isfinite(v), v, 0)
    o[live] = (p @ vv)[live]
    eo = (p * (BF16 + ez + 2.0 ** -20)) @ np.abs(vv) + (p @ np.abs(vv)) * (worst + n * 2.0 ** -23)[:, None]
    return o, lse, eo, el


def causal(rows, keys, first=0):
    return np.arange(keys)[None] <= first + np.arange(rows)[:, None]


def attend_grad(q, k, v, scale, o, lse, do):
    """One head of one sequence, causal, given the stored o and lse: dict name -> (value, bound)."""
    q, k, v, o, lse, do = (np.asarray(t, dtype=np.float64) for t in (q, k, v, o, lse, do))
    n, D = q.shape
    seen = causal(n, n)
    z, ez = scores(q, k, scale)
    with np.errstate(over="ignore"):
        p = np.where(seen, np.exp(np.where(seen, z - lse[:, None], 0)), 0)
    ep = p * (ez + np.abs(lse)[:, None] * 2.0 ** -22 + 2.0 ** -20)
    dp, delta = do @ v.T, (do * o).sum(1, keepdims=True)
    edp = (D + 2) * 2.0 ** -23 * (np.abs(do) @ np.abs(v).T + (np.abs(do) * np.abs(o)).sum(1, keepdims=True))
    ds = p * (dp - delta)
    eds = ep * np.abs(dp - delta) + p * edp + np.abs(ds) * (BF16 + 2.0 ** -21)
    total = (n + 4) * 2.0 ** -23

    def product(a, ea, b):
        return a @ b, ea @ np.abs(b) + total * (np.abs(a) @ np.abs(b))
    dv = product(p.T, (ep + p * BF16).T, do)
    dq, dk = product(ds, eds, k), product(ds.T, eds.T, q)
    s = abs(scale)
    return {"dq": (scale * dq[0], s * dq[1]), "dk": (scale * dk[0], s * dk[1]), "dv": dv}
