"""Cases of the gated recurrence (scan, its gradients, decode) and of the RMS norm beside it.

``run`` computes a case in its plain form (elementary torch operations in 32 bits) or, with ``own``
set, through the framework's entry points; ``exact`` computes it from the definition in 64 bits.
"""
import math

import numpy as np
import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
EPS = 1e-5


# ------------------------------------------------------------------------------------------ cases
def _scan(name, op, B, T, C, dtype="bf16", packed=0, pool=0, fused=False, state=True):
    """A scan over B sequences of T tokens, or (``packed`` > 0) over B sequences of random lengths of
    at most T tokens drawn with that number; ``pool`` slots of states, some sequences padded;
    ``fused``: x, r, g are column ranges of one projection's output."""
    c = {"op": op, "B": B, "T": T, "C": C, "dtype": dtype, "packed": packed, "pool": pool, "fused": fused,
         "state": state}
    return {"name": name, **c} if name else c


def _decode(name, B, T, C, pool, dtype="bf16", fused=False):
    c = {"op": "decode", "B": B, "T": T, "C": C, "dtype": dtype, "pool": pool, "fused": fused}
    return {"name": name, **c} if name else c


def _norm(name, op, rows, C, dtype="bf16", residual=True, out="same"):
    c = {"op": op, "rows": rows, "C": C, "dtype": dtype, "residual": residual, "out": out}
    return {"name": name, **c} if name else c


def listed():
    return [
        # a short prompt of a small layer (4 heads of 128 channels): latency
        _scan("scan fwd T=256", "scan_fwd", 1, 256, 512),
        # a training batch of a wide layer (64 heads of 128), states carried from the batch before
        _scan("scan fwd 2x8192", "scan_fwd", 2, 8192, 8192),
        # a serving batch of prompts of random lengths, states in a pool, some requests padded
        _scan("scan fwd packed", "scan_fwd", 32, 4096, 4096, packed=7, pool=64),
        # one long document, few and odd channels, FP32 activations out of one fused projection
        _scan("scan fwd long", "scan_fwd", 1, 131071, 500, dtype="fp32", fused=True),
        # the gradients of the training batch, written into the projections' own layout
        _scan("scan bwd 2x8192", "scan_bwd", 2, 8192, 8192, fused=True),
        # the gradients of a packed batch with an odd channel count
        _scan("scan bwd packed", "scan_bwd", 24, 2048, 1001, packed=11, pool=40),
        # one token per request over a pool of states: the serving step
        _decode("decode T=1", 128, 1, 8192, 256),
        # eight draft tokens per request
        _decode("decode T=8", 128, 8, 8192, 256, fused=True),
        # the norm before a layer in the serving step
        _norm("norm fwd 128 rows", "norm_fwd", 128, 8192),
        # the norm before a prompt's projections, with 8-bit rows and their scales
        _norm("norm fwd fp8", "norm_fwd", 16384, 8192, out="fp8_row"),
        # the norm's gradients in training
        _norm("norm bwd 16384 rows", "norm_bwd", 16384, 4096),
        # the same for odd sizes
        _norm("norm bwd odd", "norm_bwd", 4099, 1001, residual=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["scan_fwd", "scan_fwd", "scan_bwd", "decode", "norm_fwd", "norm_bwd"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    C = _log(rng, 64, 8192)
    if rng.random() < 0.5:
        C = max(64, C // 128 * 128)
    most = (1 << 26) if dtype == "bf16" else (1 << 25)  # elements
    if op in ("scan_fwd", "scan_bwd"):
        packed = rng.randrange(1, 1000) if rng.random() < 0.5 else 0
        B = _log(rng, 1, 64)
        T = _log(rng, 1, max(1, min(131072, most // (B * C))))
        return _scan(None, op, B, T, C, dtype, packed, B + rng.randrange(0, 64) if rng.random() < 0.6 else 0,
                     rng.random() < 0.4, rng.random() < 0.8)
    if op == "decode":
        B = _log(rng, 1, 256)
        return _decode(None, B, rng.randrange(1, 9), C, B + rng.randrange(0, 128), dtype, rng.random() < 0.4)
    rows = _log(rng, 1, min(16384, most // C))
    out = rng.choice(["same", "fp8_row", "fp8_128"]) if op == "norm_fwd" else "same"
    return _norm(None, op, rows, C, dtype, rng.random() < 0.7, out)


# ----------------------------------------------------------------------------------------- inputs
def _lengths(case):
    """Lengths of the sequences (host), from the case alone."""
    if case["packed"]:
        n = np.random.RandomState(case["packed"]).randint(0, case["T"] + 1, case["B"])
        n[0] = case["T"]
        return [int(v) for v in n]
    return [case["T"]] * case["B"]


def _slots(case):
    """The pool slot of each sequence, negative for a padded one; None without a pool."""
    if not case["pool"]:
        return None
    r = np.random.RandomState(case["pool"])
    idx = r.permutation(case["pool"])[: case["B"]].astype(np.int32)
    idx[r.permutation(case["B"])[: case["B"] // 8]] = -1
    return idx


def _gates(case, tokens, gen, dev):
    """x, r, g: [tokens, C], apart or as column ranges of one [tokens, 3 C] projection."""
    C, dt = case["C"], TYPES[case["dtype"]]
    if case["fused"]:
        xrg = torch.randn((tokens, 3 * C), generator=gen, device=dev).to(dt)
        return xrg[:, :C], xrg[:, C:2 * C], xrg[:, 2 * C:]
    return tuple(torch.randn((tokens, C), generator=gen, device=dev).to(dt) for _ in range(3))


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    op, C, dt = case["op"], case["C"], TYPES[case["dtype"]]
    s = {"case": case}
    if op in ("norm_fwd", "norm_bwd"):
        rows = case["rows"]

        def rand(scale):
            return (torch.randn((rows, C), generator=gen, device=dev) * scale).to(dt)

        s["x"] = rand(1.0)
        s["w"] = 1 + 0.1 * torch.randn(C, generator=gen, device=dev)
        if op == "norm_fwd":
            s["res"] = rand(2.0) if case["residual"] else None
        else:
            s["dy"] = rand(1.0)
            s["dres"] = rand(1.0) if case["residual"] else None
        return s
    # decays spread as the framework's slopes are: exp(-1) to exp(-1 / 256) for an open gate
    s["slopes"] = torch.exp2(-8.0 * torch.arange(1, C + 1, device=dev, dtype=torch.float32) / C)
    if op == "decode":
        s["x"], s["r"], s["g"] = _gates(case, case["B"] * case["T"], gen, dev)
        s["state"] = torch.randn((case["pool"], C), generator=gen, device=dev)
        idx = _slots(case)
        s["idx"], s["live"] = torch.from_numpy(idx).to(dev), torch.from_numpy(np.nonzero(idx >= 0)[0]).to(dev)
        s["slot"] = torch.from_numpy(idx[idx >= 0].astype(np.int64)).to(dev)
        s["o"] = torch.zeros((case["B"] * case["T"], C), dtype=dt, device=dev)
        return s
    lens = _lengths(case)
    tokens = sum(lens)
    s["x"], s["r"], s["g"] = _gates(case, tokens, gen, dev)
    idx = _slots(case)
    slots = np.arange(case["B"]) if idx is None else idx
    cu = np.concatenate([[0], np.cumsum(lens)])
    s["cu"] = torch.from_numpy(cu.astype(np.int32)).to(dev) if case["packed"] else None
    s["idx"] = None if idx is None else torch.from_numpy(idx).to(dev)
    pool = case["pool"] or case["B"]
    # the batch's rows, as a program that packs it knows them: first and last rows and slots of the
    # sequences that run, and the rows of padded sequences
    run_ = [n for n in range(case["B"]) if slots[n] >= 0]
    full = [n for n in run_ if lens[n] > 0]
    s["first"] = torch.tensor([int(cu[n]) for n in full], dtype=torch.int64, device=dev)
    s["last"] = torch.tensor([int(cu[n + 1]) - 1 for n in full], dtype=torch.int64, device=dev)
    s["slot"] = torch.tensor([int(slots[n]) for n in full], dtype=torch.int64, device=dev)
    s["empty"] = torch.tensor([int(slots[n]) for n in run_ if lens[n] == 0], dtype=torch.int64, device=dev)
    dead = np.zeros(tokens, dtype=bool)
    for n in range(case["B"]):
        dead[cu[n]:cu[n + 1]] = slots[n] < 0
    s["dead"] = torch.from_numpy(dead).to(dev) if dead.any() else None
    s["h0"] = torch.randn((pool, C), generator=gen, device=dev) if case["state"] else None

    def zeros():
        return torch.zeros((tokens, C), dtype=dt, device=dev)

    if op == "scan_fwd":
        s["o"] = zeros()
        s["hf"] = torch.zeros((pool, C), device=dev)
        return s
    lam, b = _terms(s["x"], s["r"], s["g"], s["slopes"])[:2]
    s["o"] = _kept(_chain(lam, b, s["first"], _start(s)), s["dead"]).to(dt)
    del lam, b
    s["dout"] = torch.randn((tokens, C), generator=gen, device=dev).to(dt)
    s["dhf"] = torch.randn((pool, C), generator=gen, device=dev) if case["state"] else None
    s["dh0"] = torch.zeros((pool, C), device=dev) if case["state"] else None
    if case["fused"]:
        d = torch.zeros((tokens, 3 * C), dtype=dt, device=dev)
        s["dx"], s["dr"], s["dg"] = d[:, :C], d[:, C:2 * C], d[:, 2 * C:]
    else:
        s["dx"], s["dr"], s["dg"] = zeros(), zeros(), zeros()
    return s


# ------------------------------------------------------------------------------------ plain forms
def _sigmoid(z):
    return 1 / (1 + torch.exp(-z))


def _terms(x, r, g, slopes):
    """Decay, input and the gates of the recurrence h_t = lam_t h_{t-1} + b_t."""
    sr, sg = _sigmoid(r.float()), _sigmoid(g.float())
    u = slopes * sr
    beta = torch.sqrt(-torch.expm1(-2 * u))
    return torch.exp(-u), beta * sg * x.float(), sr, sg, u, beta


def _linear(a, b):
    """h_t = a_t h_{t-1} + b_t along the first axis, by pairs of steps."""
    n = a.shape[0]
    if n == 1:
        return b
    m = n // 2
    a0, b0, a1, b1 = a[0:2 * m:2], b[0:2 * m:2], a[1::2], b[1::2]
    odd = _linear(a1 * a0, a1 * b0 + b1)
    h = torch.empty_like(b)
    h[1::2] = odd
    h[0] = b[0]
    h[2::2] = a[2::2] * odd[: (n - 1) // 2] + b[2::2]
    return h


def _chain(lam, b, first, start):
    """The recurrence over packed sequences: rows ``first`` start one, from the states ``start``."""
    if not lam.shape[0]:
        return b
    b = b.index_put((first,), b[first] + lam[first] * start)
    return _linear(lam.index_fill(0, first, 0.0), b)


def _start(s):
    return s["h0"][s["slot"]] if s["h0"] is not None else s["slopes"].new_zeros((s["slot"].shape[0], s["case"]["C"]))


def _kept(v, dead):
    return v if dead is None else v.masked_fill(dead[:, None], 0.0)


def _plain_scan(s):
    lam, b = _terms(s["x"], s["r"], s["g"], s["slopes"])[:2]
    h = _chain(lam, b, s["first"], _start(s))
    hf = torch.zeros_like(s["hf"])
    hf[s["slot"]] = h[s["last"]]
    if s["h0"] is not None:
        hf[s["empty"]] = s["h0"][s["empty"]]
    return {"o": _kept(h, s["dead"]).to(s["o"].dtype), "h_final": hf}


def _plain_scan_bwd(s):
    x = s["x"].float()
    lam, _, sr, sg, u, beta = _terms(s["x"], s["r"], s["g"], s["slopes"])
    dout = s["dout"].float()
    if s["dhf"] is not None:
        dout = dout.index_put((s["last"],), dout[s["last"]] + s["dhf"][s["slot"]])
    # w_t = lam_t (dout_t + w_{t+1}) runs from the last token of each sequence to its first
    if x.shape[0]:
        w = _linear((lam.index_fill(0, s["last"], 0.0)).flip(0), (lam * dout).flip(0)).flip(0)
        after = torch.cat([w[1:], torch.zeros_like(w[:1])]).index_fill(0, s["last"], 0.0)
        before = torch.cat([s["o"][:1], s["o"][:-1]]).float().index_put((s["first"],), _start(s))
    else:
        w = after = before = x
    G = dout + after
    dx = G * beta * sg
    dg = G * beta * x * sg * (1 - sg)
    du = G * (sg * x * torch.where(u > 0, lam * lam / beta, 0.0) - lam * before)
    dr = du * u * (1 - sr)
    dt = s["x"].dtype
    out = {"dx": _kept(dx, s["dead"]).to(dt), "dr": _kept(dr, s["dead"]).to(dt), "dg": _kept(dg, s["dead"]).to(dt),
           "dslopes": _kept(du * sr, s["dead"]).sum(0)}
    if s["dh0"] is not None:
        dh0 = torch.zeros_like(s["dh0"])
        dh0[s["slot"]] = w[s["first"]]
        dh0[s["empty"]] = s["dhf"][s["empty"]]
        out["dh0"] = dh0
    return out


def _plain_decode(s):
    B, T, C = s["case"]["B"], s["case"]["T"], s["case"]["C"]
    lam, b = (v.view(B, T, C)[s["live"]].transpose(0, 1) for v in _terms(s["x"], s["r"], s["g"], s["slopes"])[:2])
    b = torch.cat([(b[0] + lam[0] * s["state"][s["slot"]])[None], b[1:]])
    h = _linear(lam, b)
    s["state"][s["slot"]] = h[-1]
    s["o"].view(B, T, C)[s["live"]] = h.transpose(0, 1).to(s["o"].dtype)
    return {"o": s["o"], "state": s["state"]}


def _plain_norm(s):
    case, x = s["case"], s["x"].float()
    t = x if s["res"] is None else x + s["res"].float()
    y = t * torch.rsqrt(t.square().mean(1, keepdim=True) + EPS) * s["w"]
    out = {} if s["res"] is None else {"residual": t.to(s["x"].dtype)}
    if case["out"] == "same":
        return {"y": y.to(s["x"].dtype), **out}
    C = case["C"]
    width = C if case["out"] == "fp8_row" else 128
    groups = -(-C // width)
    p = torch.nn.functional.pad(y, (0, groups * width - C)).view(-1, groups, width)
    scales = p.abs().amax(2).clamp_min(2.0 ** -40) / 448
    q = (p / scales[:, :, None]).reshape(-1, groups * width)[:, :C]
    return {"y": q.clamp(-448, 448).to(torch.float8_e4m3fn), "scales": scales, **out}


def _plain_norm_bwd(s):
    t, dy, w = s["x"].float(), s["dy"].float(), s["w"]
    rstd = torch.rsqrt(t.square().mean(1, keepdim=True) + EPS)
    n, wdy = t * rstd, w * dy
    dx = rstd * (wdy - n * (wdy * n).mean(1, keepdim=True))
    if s["dres"] is not None:
        dx = dx + s["dres"].float()
    return {"dx": dx.to(s["x"].dtype), "dweight": (dy * n).sum(0)}


# --------------------------------------------------------------------------------- the framework's
def _own_scan(s):
    import linear_attention_prefill_chunkwise_gb300 as lap
    lap.la_gated_scan_fwd(s["x"], s["r"], s["g"], s["slopes"], h0=s["h0"], state_indices=s["idx"],
                          cu_seqlens=s["cu"], o=s["o"], h_final=s["hf"],
                          seq_len=None if s["case"]["packed"] else s["case"]["T"])
    return {"o": s["o"], "h_final": s["hf"]}


def _own_scan_bwd(s):
    import linear_attention_prefill_chunkwise_gb300 as lap
    dx, dr, dg, dslopes, dh0 = lap.la_gated_scan_bwd(
        s["x"], s["r"], s["g"], s["slopes"], s["o"], s["dout"], h0=s["h0"], dh_final=s["dhf"],
        state_indices=s["idx"], cu_seqlens=s["cu"], dx=s["dx"], dr=s["dr"], dg=s["dg"], dh0=s["dh0"],
        seq_len=None if s["case"]["packed"] else s["case"]["T"])
    out = {"dx": dx, "dr": dr, "dg": dg, "dslopes": dslopes}
    return out if dh0 is None else {**out, "dh0": dh0}


def _own_decode(s):
    import linear_attention_prefill_chunkwise_gb300 as lap
    lap.la_gated_decode(s["x"], s["r"], s["g"], s["slopes"], s["state"], s["case"]["T"], state_indices=s["idx"],
                        o=s["o"])
    return {"o": s["o"], "state": s["state"]}


def _own_norm(s):
    import linear_attention_prefill_chunkwise_gb300 as lap
    if s["case"]["out"] == "same":
        y, t = lap.la_rms_norm_fwd(s["x"], s["w"], EPS, residual=s["res"])
        out = {"y": y}
    else:
        y, scales, t = lap.la_rms_norm_fwd_fp8(s["x"], s["w"], EPS, residual=s["res"],
                                               group=0 if s["case"]["out"] == "fp8_row" else 128)
        out = {"y": y, "scales": scales}
    return out if s["res"] is None else {**out, "residual": t}


def _own_norm_bwd(s):
    import linear_attention_prefill_chunkwise_gb300 as lap
    dx, dweight = lap.la_rms_norm_bwd(s["x"], s["w"], EPS, s["dy"], dres=s["dres"])
    return {"dx": dx, "dweight": dweight}


PLAIN = {"scan_fwd": _plain_scan, "scan_bwd": _plain_scan_bwd, "decode": _plain_decode, "norm_fwd": _plain_norm,
         "norm_bwd": _plain_norm_bwd}
OWN = {"scan_fwd": _own_scan, "scan_bwd": _own_scan_bwd, "decode": _own_decode, "norm_fwd": _own_norm,
       "norm_bwd": _own_norm_bwd}


def run(state):
    return (OWN if own else PLAIN)[state["case"]["op"]](state)


# ------------------------------------------------------------------------------------------- work
def work(case):
    op, C, e = case["op"], case["C"], 2 if case["dtype"] == "bf16" else 4
    if op == "norm_fwd":
        n = case["rows"] * C
        out = e if case["out"] == "same" else 1
        scales = 0 if case["out"] == "same" else 4 * case["rows"] * (1 if case["out"] == "fp8_row" else -(-C // 128))
        return {"bytes": n * (e * (3 if case["residual"] else 1) + out) + scales + 4 * C, "flops": 5 * n}
    if op == "norm_bwd":
        n = case["rows"] * C
        return {"bytes": n * e * (4 if case["residual"] else 3) + 8 * C, "flops": 12 * n}
    idx = _slots(case)
    if op == "decode":
        live = int((idx >= 0).sum())
        return {"bytes": live * C * (4 * e * case["T"] + 8) + 4 * C, "flops": 25 * live * case["T"] * C}
    lens = _lengths(case)
    live = [lens[n] for n in range(case["B"]) if idx is None or idx[n] >= 0]
    n, states = sum(live) * C, len(live) * C * 4
    if op == "scan_fwd":
        return {"bytes": 4 * e * n + states * (2 if case["state"] else 1) + 4 * C, "flops": 25 * n}
    return {"bytes": 8 * e * n + states * (3 if case["state"] else 0) + 8 * C, "flops": 45 * n}


# ------------------------------------------------------------------------------------------ exact
def _exact_gates(s):
    x, r, g = (s[k].double() for k in ("x", "r", "g"))
    a, i = torch.sigmoid(r), torch.sigmoid(g)
    u = s["slopes"].double() * a
    return x, a, i, u, torch.exp(-u), torch.sqrt(-torch.expm1(-2 * u))


def _sequences(case):
    """(first row, rows, slot) of the sequences that run."""
    lens, idx = _lengths(case), _slots(case)
    cu = np.concatenate([[0], np.cumsum(lens)])
    slots = np.arange(case["B"]) if idx is None else idx
    return [(int(cu[n]), lens[n], int(slots[n])) for n in range(case["B"]) if slots[n] >= 0]


def _by_steps(case):
    """Row numbers of the sequences' t-th tokens for each t, longest sequences first."""
    seqs = sorted(_sequences(case), key=lambda q: -q[1])
    at = torch.tensor([q[0] for q in seqs], device="cuda")
    counts = np.searchsorted(-np.array([q[1] for q in seqs]), -np.arange(case["T"]), side="left") if seqs else []
    return seqs, at, [int(v) for v in counts]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm_fwd":
        t = s["x"].double() + (0 if s["res"] is None else s["res"].double())
        y = t / (t.pow(2).sum(1, keepdim=True) / case["C"] + EPS).sqrt() * s["w"].double()
        out = {} if s["res"] is None else {"residual": t}
        if case["out"] == "same":
            return {"y": y, **out}
        width = case["C"] if case["out"] == "fp8_row" else 128
        parts = y.split(width, 1)
        scales = torch.stack([p.abs().amax(1).clamp_min(2.0 ** -40) / 448 for p in parts], 1)
        return {"y": torch.cat([p / scales[:, k, None] for k, p in enumerate(parts)], 1), "scales": scales, **out}
    if op == "norm_bwd":
        t = s["x"].double().requires_grad_()
        w = s["w"].double().requires_grad_()
        y = t / (t.pow(2).sum(1, keepdim=True) / case["C"] + EPS).sqrt() * w
        y.backward(s["dy"].double())
        dx = t.grad if s["dres"] is None else t.grad + s["dres"].double()
        return {"dx": dx, "dweight": w.grad}
    x, a, i, u, lam, beta = _exact_gates(s)
    b = beta * i * x
    if op == "decode":
        o, state = torch.zeros_like(b), s["state"].double()
        h = state[s["slot"]]
        for t in range(case["T"]):
            rows = s["live"] * case["T"] + t
            h = lam[rows] * h + b[rows]
            o[rows] = h
        state[s["slot"]] = h
        return {"o": o, "state": state}
    if case["T"] > 200000:
        return None
    seqs, at, counts = _by_steps(case)
    slot = torch.tensor([q[2] for q in seqs], device="cuda", dtype=torch.int64)
    pool = case["pool"] or case["B"]
    h0 = s["h0"].double()[slot] if s["h0"] is not None else torch.zeros((len(seqs), case["C"]), dtype=torch.float64,
                                                                        device="cuda")
    if op == "scan_fwd":
        o, h = torch.zeros_like(b), h0.clone()
        for t, k in enumerate(counts):
            rows = at[:k] + t
            h[:k] = lam[rows] * h[:k] + b[rows]
            o[rows] = h[:k]
        hf = torch.zeros((pool, case["C"]), dtype=torch.float64, device="cuda")
        hf[slot] = h
        return {"o": o, "h_final": hf}
    G = torch.zeros_like(b)
    g = s["dhf"].double()[slot] if s["dhf"] is not None else torch.zeros_like(h0)  # dL/dh after the token
    dout, before = s["dout"].double(), torch.zeros_like(b)
    o = s["o"].double()
    for t in range(len(counts) - 1, -1, -1):
        k = counts[t]
        rows = at[:k] + t
        G[rows] = dout[rows] + g[:k]
        before[rows] = h0[:k] if t == 0 else o[rows - 1]
        g[:k] = lam[rows] * G[rows]
    du = G * (i * x * lam * lam / beta - lam * before)
    out = {"dx": G * beta * i, "dr": du * u * (1 - a), "dg": G * b * (1 - i), "dslopes": (du * a).sum(0)}
    if s["dh0"] is not None:
        dh0 = torch.zeros((pool, case["C"]), dtype=torch.float64, device="cuda")
        dh0[slot] = g
        out["dh0"] = dh0
    return out
