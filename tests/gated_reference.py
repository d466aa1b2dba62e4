"""Plain 64-bit forms of the gated recurrence and of the RMS norm (numpy, token by token), each
with a bound on the FP32 kernels' error computed alongside.

The bounds count what the kernels do in FP32: a rounding is 2^-24 relative, the hardware's exp2
and reciprocal 2^-22 at most each, an exponent's argument rounding |z| 2^-23.  Hence, relative,
    sigmoid          e_s(z) = 2^-21 + |z| 2^-23
    lambda = e^-u    d(u)   = u (e_s + 2^-21) + 2^-24 for u < 1/4 (series), u e_s + 2^-21 beyond
    beta             e_s(r) + 2^-19 (1 - lambda^2 without cancellation, rsqrt 2^-22)
and along the recurrence h = lambda h + b, with M the same recurrence on absolute values,
    E_t = lambda (E_{t-1} + d M_{t-1}) + e_b |b_t| + 2^-22 M_t
(2^-22: the products of lambdas and the sums of a blocked evaluation, two roundings each way).
The output's own rounding adds half a step of its type.
"""
from __future__ import annotations

import numpy as np

HALF_STEP = {"bf16": 2.0 ** -8, "fp32": 2.0 ** -24, "e4m3": 2.0 ** -4}


def sigmoid(z):
    return np.where(z >= 0, 1 / (1 + np.exp(-np.abs(z))), np.exp(-np.abs(z)) / (1 + np.exp(-np.abs(z))))


def gates(x, r, g, slopes):
    sr, sg = sigmoid(r), sigmoid(g)
    u = slopes * sr
    lam, beta = np.exp(-u), np.sqrt(-np.expm1(-2 * u))
    return sr, sg, u, lam, beta


def gate_errors(r, g, u):
    zr, zg = (np.where(np.isfinite(z), np.abs(z), 0) for z in (r, g))
    er, eg = 2.0 ** -21 + zr * 2.0 ** -23, 2.0 ** -21 + zg * 2.0 ** -23
    d = np.where(u < 0.25, u * (er + 2.0 ** -21) + 2.0 ** -24, u * er + 2.0 ** -21)
    return er, eg, d, er + 2.0 ** -19


def scan_one(x, r, g, slopes, h0):
    """One sequence [L, C] from h0 [C]: (o, h_final, bound of o, bound of h_final), in 64 bits."""
    x, r, g, slopes = (np.asarray(v, dtype=np.float64) for v in (x, r, g, slopes))
    _, sg, u, lam, beta = gates(x, r, g, slopes)
    b = beta * sg * x
    er, eg, d, eb = gate_errors(r, g, u)
    h = np.array(h0, dtype=np.float64)
    M, E = np.abs(h), np.zeros_like(h)
    o, bound = np.empty_like(b), np.empty_like(b)
    for t in range(x.shape[0]):
        E = lam[t] * (E + d[t] * M)
        h = lam[t] * h + b[t]
        M = lam[t] * M + np.abs(b[t])
        E = E + (eb[t] + eg[t] + 2.0 ** -22) * np.abs(b[t]) + 2.0 ** -22 * M
        o[t], bound[t] = h, E
    return o, h, bound, E


def grad_one(x, r, g, slopes, h0, o, dout, dhf):
    """Gradients of one sequence given the forward's stored output o: dict name -> (value, bound);
    "ds" holds the sequence's sum of the terms of dslopes."""
    x, r, g, slopes, o, dout = (np.asarray(v, dtype=np.float64) for v in (x, r, g, slopes, o, dout))
    L = x.shape[0]
    sr, sg, u, lam, beta = gates(x, r, g, slopes)
    er, eg, d, eb = gate_errors(r, g, u)
    w = np.array(dhf, dtype=np.float64)
    M, E = np.abs(w), np.zeros_like(w)
    G, EG = np.empty_like(x), np.empty_like(x)
    for t in range(L - 1, -1, -1):
        G[t] = dout[t] + w
        Mg = np.abs(dout[t]) + M
        EG[t] = E + 2.0 ** -23 * Mg
        w = lam[t] * G[t]
        M = lam[t] * Mg
        E = lam[t] * (EG[t] + d[t] * Mg) + 2.0 ** -22 * M
    before = np.concatenate([np.asarray(h0, dtype=np.float64)[None], o[:-1]])[:L]
    with np.errstate(divide="ignore", invalid="ignore"):
        q = np.where(u > 0, lam * lam / beta, 0.0)
    dx = G * beta * sg
    edx = EG * beta * sg + np.abs(dx) * (eb + eg + 2.0 ** -21)
    dg = dx * x * (1 - sg)
    edg = edx * np.abs(x) * (1 - sg) + np.abs(dx * x) * (sg * eg + 2.0 ** -23)
    a1, a2 = sg * x * q, lam * before
    du = G * (a1 - a2)
    size = np.abs(G) * (np.abs(a1) + np.abs(a2))
    edu = EG * (np.abs(a1) + np.abs(a2)) + size * (eb + eg + 2 * d + 2.0 ** -20)
    dr = du * u * (1 - sr)
    edr = edu * u * (1 - sr) + np.abs(du) * u * ((1 - sr) * (er + 2.0 ** -22) + sr * er + 2.0 ** -23)
    ds = du * sr
    eds = edu * sr + np.abs(ds) * (er + 2.0 ** -23)
    return {"dx": (dx, edx), "dr": (dr, edr), "dg": (dg, edg), "dh0": (w, E),
            "ds": (ds.sum(0), eds.sum(0) + L * 2.0 ** -24 * np.abs(ds).sum(0))}


def norm(x, residual, weight, eps):
    """(y, s, bound of y): s = x + residual, y = s / sqrt(mean(s^2) + eps) * weight.  The sum of C
    squares has C 2^-24 relative error at most; the mean, rsqrt (2^-22) and two products follow."""
    s = np.asarray(x, dtype=np.float64) + (0 if residual is None else np.asarray(residual, dtype=np.float64))
    C = s.shape[1]
    y = s / np.sqrt((s * s).mean(1, keepdims=True) + eps) * weight
    return y, s, np.abs(y) * (0.5 * C * 2.0 ** -24 + 2.0 ** -21) + 2.0 ** -23 * np.abs(y)


def norm_grad(s, weight, eps, dy, dres):
    """dict name -> (value, bound) of the norm's gradients."""
    s, dy = np.asarray(s, dtype=np.float64), np.asarray(dy, dtype=np.float64)
    rows, C = s.shape
    rstd = 1 / np.sqrt((s * s).mean(1, keepdims=True) + eps)
    n, wdy = s * rstd, weight * dy
    m = (wdy * n).mean(1, keepdims=True)
    dx = rstd * (wdy - n * m)
    e = 0.5 * C * 2.0 ** -24 + 2.0 ** -21  # relative error of rstd and n
    edot = np.abs(wdy * n).mean(1, keepdims=True) * (C * 2.0 ** -24 + 2 * e)
    edx = rstd * (np.abs(wdy) * e + np.abs(n) * edot + np.abs(n * m) * 3 * e + 2.0 ** -22 * (np.abs(wdy) + np.abs(n * m)))
    if dres is not None:
        dx = dx + np.asarray(dres, dtype=np.float64)
        edx = edx + 2.0 ** -23 * np.abs(dx)
    t = np.abs(dy * n).sum(0)
    return {"dx": (dx, edx), "dweight": ((dy * n).sum(0), t * (e + (rows + 2) * 2.0 ** -24))}
