"""Cases of the softmax-attention layers beside the linear ones: norm and rotation of queries and
keys, attention over whole prompts and its gradients, attention of drafted tokens over a cache, and
the writes into that cache.

``run`` computes a case in its plain form (elementary torch operations in 32 bits) or, with ``own``
set, through the framework's entry points; ``exact`` computes it from the definition in 64 bits.
"""
import math

import numpy as np
import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
EPS = 1e-6
ROWS = 1024  # query rows of a sequence that the plain form takes at once


# ------------------------------------------------------------------------------------------ cases
def _rope(name, op, tokens, H, HK, D, R, dtype="bf16", pairs="halves", base=10000.0, start=0, fused=True):
    """Norm and rotation of H query and HK key heads; R of D elements rotate; positions count from
    ``start``; ``fused``: q and k are column ranges of one projection's output."""
    c = {"op": op, "tokens": tokens, "H": H, "HK": HK, "D": D, "R": R, "dtype": dtype, "pairs": pairs, "base": base,
         "start": start, "fused": fused}
    return {"name": name, **c} if name else c


def _attn(name, op, B, T, H, HK, D, packed=0, fused=False):
    """Causal attention over B sequences of T tokens, or (``packed`` > 0) of random lengths of at most
    T tokens drawn with that number."""
    c = {"op": op, "B": B, "T": T, "H": H, "HK": HK, "D": D, "packed": packed, "fused": fused}
    return {"name": name, **c} if name else c


def _verify(name, B, T, H, HK, D, S, page, lens, tree):
    """T drafted tokens of each of B requests over a cache of at most S tokens per request, in pages
    of ``page`` tokens (0: one range per request); ``lens`` draws the requests' lengths."""
    c = {"op": "verify", "B": B, "T": T, "H": H, "HK": HK, "D": D, "S": S, "page": page, "lens": lens, "tree": tree}
    return {"name": name, **c} if name else c


def _commit(name, B, T, HK, D, S, page, lens, prompt):
    """Keys and values into the cache: an accepted path of each request's T drafted tokens, or
    (``prompt``) packed prompts of at most T tokens."""
    c = {"op": "commit", "B": B, "T": T, "HK": HK, "D": D, "S": S, "page": page, "lens": lens, "prompt": prompt}
    return {"name": name, **c} if name else c


def listed():
    return [
        # the serving step of 128 requests with eight drafted tokens each, far into their texts
        _rope("norm rope fwd 128x8", "rope_fwd", 1024, 64, 8, 128, 128, base=1e6, start=100000),
        # a prompt of a wide layer, half of each head rotated
        _rope("norm rope fwd 16384", "rope_fwd", 16384, 64, 8, 128, 64),
        # the gradients of a training batch
        _rope("norm rope bwd 16384", "rope_bwd", 16384, 32, 4, 128, 128),
        # the same in FP32 for odd sizes, neighbours as pairs
        _rope("norm rope bwd odd", "rope_bwd", 4099, 12, 3, 64, 64, dtype="fp32", pairs="neighbours", fused=False),
        # a few short prompts of a small layer: latency
        _attn("attn fwd short", "attn_fwd", 4, 500, 16, 2, 64, packed=3, fused=True),
        # a training batch of a wide layer
        _attn("attn fwd 2x8192", "attn_fwd", 2, 8192, 64, 8, 128),
        # gradients of a training batch
        _attn("attn bwd 2x8192", "attn_bwd", 2, 8192, 32, 4, 128),
        # gradients of a packed batch of documents of odd lengths
        _attn("attn bwd packed", "attn_bwd", 24, 2047, 16, 16, 64, packed=11, fused=True),
        # one token per request over a paged cache of ragged lengths: the serving step
        _verify("verify T=1", 128, 1, 64, 8, 128, 8192, 64, 5, tree=False),
        # trees of 16 drafted tokens over long contexts
        _verify("verify tree T=16", 16, 16, 32, 8, 128, 32768, 16, 9, tree=True),
        # the accepted paths of the drafted trees
        _commit("commit drafts", 128, 8, 8, 128, 1024, 64, 5, prompt=False),
        # the prompts' keys and values
        _commit("commit prompts", 16, 4096, 8, 128, 8192, 64, 9, prompt=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope_fwd", "rope_bwd", "attn_fwd", "attn_fwd", "attn_bwd", "attn_bwd", "verify", "verify",
                     "commit"])
    HK = rng.choice([1, 2, 3, 4, 8])
    if op in ("rope_fwd", "rope_bwd"):
        D = rng.choice([64, 128, 256])
        H = HK * rng.choice([1, 2, 5, 8])
        dtype = rng.choice(["bf16", "bf16", "fp32"])
        most = (1 << 27) if op == "rope_fwd" else (1 << 26)
        R = rng.choice([D, D, D // 2, 2 * rng.randrange(1, D // 2 + 1)])
        return _rope(None, op, _log(rng, 1, min(16384, most // ((H + HK) * D * (2 if dtype == "fp32" else 1)))), H, HK,
                     D, R, dtype, rng.choice(["halves", "neighbours"]), rng.choice([1e4, 1e6]),
                     rng.choice([0, 100000, 3000000]), rng.random() < 0.5)
    D = rng.choice([64, 128])
    if op in ("attn_fwd", "attn_bwd"):
        T = _log(rng, 1, 16384)
        G = rng.choice([1, 2, 4, 5, 8])
        most = (1 << 32) if op == "attn_fwd" else (1 << 31)  # products of queries and keys
        H = max(1, min(HK * G, most // (T * T)))
        HK = max(k for k in (1, 2, 3, 4, 8) if k <= HK and H % k == 0)
        B = _log(rng, 1, max(1, min(32, most // (T * T * H), 32768 // T)))
        return _attn(None, op, B, T, H, HK, D, rng.randrange(1, 1000) if rng.random() < 0.5 else 0, rng.random() < 0.5)
    B = _log(rng, 1, 128)
    page = rng.choice([0, 16, 32, 64, 128])
    if op == "verify":
        S = _log(rng, 1, max(1, min(65536, (1 << 29) // (B * HK * D))))
        T = rng.choice([1, 1, 2, 3, 8, 16, 33])
        return _verify(None, B, T, HK * rng.choice([1, 2, 4, 5, 8]), HK, D, S, page, rng.randrange(1, 1000),
                       T > 1 and rng.random() < 0.6)
    prompt = rng.random() < 0.5
    T = _log(rng, 1, min(4096, 65536 // B)) if prompt else rng.randrange(1, 17)
    S = T + _log(rng, 1, max(1, min(8192, (1 << 27) // (B * HK * D))))
    return _commit(None, B, T, HK, D, S, page, rng.randrange(1, 1000), prompt)


# ----------------------------------------------------------------------------------------- inputs
def _lengths(case):
    """Lengths of an attention batch's sequences (host), from the case alone."""
    if case["packed"]:
        n = np.random.RandomState(case["packed"]).randint(0, case["T"] + 1, case["B"])
        n[0] = case["T"]
        return [int(v) for v in n]
    return [case["T"]] * case["B"]


def _cache_lengths(case):
    """Tokens in the cache of each request (host), negative for a padded request."""
    room = case["S"] - (case["T"] if case["op"] == "commit" else 0)
    r = np.random.RandomState(case["lens"])
    n = r.randint(0, room + 1, case["B"]).astype(np.int32)
    n[0] = room
    n[1:][r.permutation(case["B"] - 1)[: case["B"] // 16]] = -1
    return n


def _counts(case):
    """Tokens that each request commits (host), and the paths [B, T] through its drafted tokens."""
    r = np.random.RandomState(case["lens"] + 1)
    B, T = case["B"], case["T"]
    n = r.randint(0, T + 1, B).astype(np.int32)
    n[0] = T
    path = np.stack([np.sort(r.permutation(T)[:k].tolist() + [T] * (T - k)) for k in n]).astype(np.int32)
    return n, path


def _heads(tokens, counts, D, dtype, fused, gen, dev):
    """Tensors [tokens, heads, D], apart or as column ranges of one projection's output."""
    if fused:
        x = torch.randn((tokens, sum(counts) * D), generator=gen, device=dev).to(dtype)
        return [t.unflatten(1, (-1, D)) for t in x.split([n * D for n in counts], 1)]
    return [torch.randn((tokens, n, D), generator=gen, device=dev).to(dtype) for n in counts]


def _tree(B, T, seed):
    """Bit masks [B, T]: each token sees itself and its ancestors in a random tree."""
    r = np.random.RandomState(seed)
    bits = np.zeros((B, T), dtype=np.uint64)
    for t in range(T):
        above = r.randint(max(0, t - 4) - 1 if t < 4 else t - 4, t, B) if t else np.full(B, -1)
        bits[:, t] = np.where(above >= 0, bits[np.arange(B), np.maximum(above, 0)], 0) | np.uint64(1 << t)
    return bits.view(np.int64)


def _cache(case, gen, dev):
    """k_cache, v_cache and the page table: pages in random order, or one range per request."""
    B, HK, D, page = case["B"], case["HK"], case["D"], case["page"]
    per = -(-case["S"] // page) if page else 1
    pages, size = (B * per, page) if page else (B, case["S"])
    k, v = (torch.randn((pages, size, HK, D), generator=gen, device=dev, dtype=torch.bfloat16) for _ in range(2))
    table = None
    if page:
        table = torch.randperm(pages, generator=gen, device=dev).to(torch.int32).view(B, per)
    return k, v, table


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    op, D = case["op"], case["D"]
    s = {"case": case}
    if op in ("rope_fwd", "rope_bwd"):
        dt, n, H, HK, R = TYPES[case["dtype"]], case["tokens"], case["H"], case["HK"], case["R"]
        # a projection's output holds the values behind the queries and keys too
        s["q"], s["k"] = _heads(n, [H, HK, HK] if case["fused"] else [H, HK], D, dt, case["fused"], gen, dev)[:2]
        s["wq"], s["wk"] = (1 + 0.1 * torch.randn(D, generator=gen, device=dev) for _ in range(2))
        s["pos"] = torch.arange(case["start"], case["start"] + n, device=dev, dtype=torch.int32)
        s["freq"] = (1 / case["base"] ** (torch.arange(0, R, 2, device=dev).double() / R)).float()
        if op == "rope_bwd":
            s["dq_out"], s["dk_out"] = _heads(n, [H, HK], D, dt, False, gen, dev)
        return s
    if op in ("attn_fwd", "attn_bwd"):
        lens = _lengths(case)
        s["lens"] = lens
        H, HK, n = case["H"], case["HK"], sum(lens)
        s["q"], s["k"], s["v"] = _heads(n, [H, HK, HK], D, torch.bfloat16, case["fused"], gen, dev)
        s["cu"] = None
        if case["packed"]:
            s["cu"] = torch.from_numpy(np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)).to(dev)
        if op == "attn_bwd":
            out = _plain_attn(s)
            s["o"], s["lse"] = out["o"], out["lse"]
            s["dout"] = torch.randn((n, H, D), generator=gen, device=dev).to(torch.bfloat16)
        return s
    s["k_cache"], s["v_cache"], s["table"] = _cache(case, gen, dev)
    lens = _cache_lengths(case)
    s["lens"], s["cache_lens"] = lens, torch.from_numpy(lens).to(dev)
    B, T, HK = case["B"], case["T"], case["HK"]
    if op == "verify":
        s["q"], s["k"], s["v"] = _heads(B * T, [case["H"], HK, HK], D, torch.bfloat16, True, gen, dev)
        s["mask"] = torch.from_numpy(_tree(B, T, case["lens"])).to(dev) if case["tree"] else None
        s["o"] = torch.zeros((B * T, case["H"], D), dtype=torch.bfloat16, device=dev)
        return s
    counts, path = _counts(case)
    s["cu"] = s["accepted"] = s["path"] = None
    if case["prompt"]:
        first = np.concatenate([[0], np.cumsum(counts)])
        tokens, s["cu"] = int(first[-1]), torch.from_numpy(first.astype(np.int32)).to(dev)
    else:
        first, tokens = np.arange(B) * T, B * T
        s["accepted"], s["path"] = torch.from_numpy(counts).to(dev), torch.from_numpy(path).to(dev)
    s["k"], s["v"] = _heads(tokens, [HK, HK], D, torch.bfloat16, True, gen, dev)
    # the rows that move, as a program that made up the batch knows them
    src, req, at = [], [], []
    for b in range(B):
        if lens[b] >= 0:
            i = np.arange(counts[b])
            src.append(first[b] + (i if case["prompt"] else path[b, : counts[b]]))
            req.append(np.full(counts[b], b))
            at.append(lens[b] + i)
    s["src"], s["req"], s["at"] = (torch.from_numpy(np.concatenate(a).astype(np.int64)).to(dev) for a in (src, req, at))
    return s


# ------------------------------------------------------------------------------------ plain forms
def _pairs(y, R, pairs):
    """The rotated part of y's last axis as two halves of its pairs."""
    return (y[..., : R // 2], y[..., R // 2:R]) if pairs == "halves" else (y[..., 0:R:2], y[..., 1:R:2])


def _turn(y, cos, sin, R, pairs):
    a, b = _pairs(y, R, pairs)
    out = y.clone()
    x0, x1 = _pairs(out, R, pairs)
    x0.copy_(a * cos - b * sin)
    x1.copy_(a * sin + b * cos)
    return out


def _angles(s):
    angle = s["pos"].double()[:, None, None] * s["freq"].double()
    return torch.cos(angle).float(), torch.sin(angle).float()


def _plain_rope(s):
    c = s["case"]
    cos, sin = _angles(s)
    out = {}
    for name, w in (("q", s["wq"]), ("k", s["wk"])):
        x = s[name].float()
        y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w
        out[name] = _turn(y, cos, sin, c["R"], c["pairs"]).to(s[name].dtype)
    return out


def _plain_rope_bwd(s):
    c = s["case"]
    cos, sin = _angles(s)
    out = {}
    for name, w in (("q", s["wq"]), ("k", s["wk"])):
        x = s[name].float()
        rstd = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
        n = x * rstd
        g = _turn(s[f"d{name}_out"].float(), cos, -sin, c["R"], c["pairs"])
        wg = w * g
        out["d" + name] = (rstd * (wg - n * (wg * n).mean(-1, keepdim=True))).to(s[name].dtype)
        out["dw" + name] = (g * n).sum((0, 1))
    return out


def _blocks(lens):
    """(first row of the sequence, first and last query row within it) of the plain form's blocks."""
    lo = 0
    for n in lens:
        for i in range(0, n, ROWS):
            yield lo, i, min(n, i + ROWS)
        lo += n


def _grouped(t, HK):
    """[rows, H, D] to [HK, G * rows, D] in 32 bits."""
    rows, H, D = t.shape
    return t.float().view(rows, HK, H // HK, D).permute(1, 2, 0, 3).reshape(HK, -1, D)


def _ungrouped(t, H):
    """The inverse: [HK, G * rows, D] to [rows, H, D]."""
    HK, n, D = t.shape
    rows = n * HK // H
    return t.view(HK, H // HK, rows, D).permute(2, 0, 1, 3).reshape(rows, H, D)


def _scores(s, lo, i, j):
    """Scaled scores [HK, G, rows, keys] of a block, minus infinity above the diagonal."""
    c = s["case"]
    q = _grouped(s["q"][lo + i:lo + j], c["HK"])
    k = s["k"][lo:lo + j].float().permute(1, 2, 0)
    z = torch.matmul(q, k).view(c["HK"], -1, j - i, j) * c["D"] ** -0.5
    rows = torch.arange(i, j, device=z.device)
    return z.masked_fill_(torch.arange(j, device=z.device) > rows[:, None], -math.inf)


def _plain_attn(s):
    c = s["case"]
    o = torch.empty(s["q"].shape, dtype=torch.bfloat16, device=s["q"].device)
    lse = torch.empty((c["H"], o.shape[0]), device=o.device)
    for lo, i, j in _blocks(s["lens"]):
        z = _scores(s, lo, i, j)
        top = z.amax(-1, keepdim=True)
        p = z.sub_(top).exp_()
        total = p.sum(-1, keepdim=True)
        v = s["v"][lo:lo + j].float().transpose(0, 1)
        out = torch.matmul(p.flatten(1, 2), v) / total.flatten(1, 2)
        o[lo + i:lo + j] = _ungrouped(out, c["H"]).to(o.dtype)
        lse[:, lo + i:lo + j] = (top + torch.log(total)).view(c["H"], j - i)
    return {"o": o, "lse": lse}


def _plain_attn_bwd(s):
    c = s["case"]
    HK, D = c["HK"], c["D"]
    dq = torch.empty(s["q"].shape, dtype=torch.bfloat16, device=s["q"].device)
    dk = torch.zeros(s["k"].shape, device=dq.device)
    dv = torch.zeros(s["v"].shape, device=dq.device)
    for lo, i, j in _blocks(s["lens"]):
        z = _scores(s, lo, i, j)
        p = z.sub_(s["lse"][:, lo + i:lo + j].view(HK, -1, j - i, 1)).exp_().flatten(1, 2)
        do, o = _grouped(s["dout"][lo + i:lo + j], HK), _grouped(s["o"][lo + i:lo + j], HK)
        dv[lo:lo + j] += torch.matmul(p.transpose(1, 2), do).transpose(0, 1)
        dp = torch.matmul(do, s["v"][lo:lo + j].float().permute(1, 2, 0))
        ds = p.mul_(dp.sub_((do * o).sum(-1, keepdim=True)))
        dq[lo + i:lo + j] = _ungrouped(torch.matmul(ds, s["k"][lo:lo + j].float().transpose(0, 1)) * D ** -0.5,
                                       c["H"]).to(dq.dtype)
        dk[lo:lo + j] += torch.matmul(ds.transpose(1, 2), _grouped(s["q"][lo + i:lo + j], HK)).transpose(0, 1) * D ** -0.5
    return {"dq": dq, "dk": dk.to(torch.bfloat16), "dv": dv.to(torch.bfloat16)}


def _cached(s, name, b, n):
    """The first n rows [n, HK, D] of request b's cache."""
    cache = s[name]
    if s["table"] is None:
        return cache[b, :n]
    page = cache.shape[1]
    return cache[s["table"][b, : -(-n // page)].long()].flatten(0, 1)[:n]


def _plain_verify(s):
    c = s["case"]
    T, H, HK = c["T"], c["H"], c["HK"]
    steps = torch.arange(T, device=s["q"].device)
    for b in range(c["B"]):
        n = int(s["lens"][b])
        if n < 0:
            continue
        rows = slice(b * T, (b + 1) * T)
        k = torch.cat([_cached(s, "k_cache", b, n), s["k"][rows]]).float().permute(1, 2, 0)
        v = torch.cat([_cached(s, "v_cache", b, n), s["v"][rows]]).float().transpose(0, 1)
        z = torch.matmul(_grouped(s["q"][rows], HK), k).view(HK, -1, T, n + T) * c["D"] ** -0.5
        if s["mask"] is None:
            seen = steps[None, :] <= steps[:, None]
        else:
            seen = (s["mask"][b][:, None] >> steps & 1) != 0
        z[..., n:].masked_fill_(~seen, -math.inf)
        p = torch.exp(z - z.amax(-1, keepdim=True))
        out = torch.matmul(p.flatten(1, 2), v) / p.sum(-1, keepdim=True).flatten(1, 2)
        s["o"][rows] = _ungrouped(out, H).to(s["o"].dtype)
    return {"o": s["o"]}


def _plain_commit(s):
    page = s["k_cache"].shape[1]
    p = s["req"] if s["table"] is None else s["table"][s["req"], s["at"] // page].long()
    for name in ("k", "v"):
        s[name + "_cache"][p, s["at"] % page] = s[name][s["src"]]
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"]}


# --------------------------------------------------------------------------------- the framework's
def _own_rope(s):
    import linear_attention_prefill_chunkwise_gb300 as lap
    q, k = lap.la_qk_norm_rope_fwd(s["q"], s["k"], s["wq"], s["wk"], EPS, s["pos"], s["freq"],
                                   interleaved=s["case"]["pairs"] == "neighbours")
    return {"q": q, "k": k}


def _own_rope_bwd(s):
    import linear_attention_prefill_chunkwise_gb300 as lap
    dq, dk, dwq, dwk = lap.la_qk_norm_rope_bwd(s["q"], s["k"], s["wq"], s["wk"], EPS, s["dq_out"], s["dk_out"], s["pos"],
                                               s["freq"], interleaved=s["case"]["pairs"] == "neighbours")
    return {"dq": dq, "dwq": dwq, "dk": dk, "dwk": dwk}


def _own_attn(s):
    import linear_attention_prefill_chunkwise_gb300 as lap
    c = s["case"]
    o, lse = lap.la_attn_prefill_fwd(s["q"], s["k"], s["v"], c["D"] ** -0.5, cu_seqlens=s["cu"],
                                     seq_len=None if c["packed"] else c["T"])
    return {"o": o, "lse": lse}


def _own_attn_bwd(s):
    import linear_attention_prefill_chunkwise_gb300 as lap
    c = s["case"]
    dq, dk, dv = lap.la_attn_prefill_bwd(s["q"], s["k"], s["v"], c["D"] ** -0.5, s["o"], s["lse"], s["dout"],
                                         cu_seqlens=s["cu"], seq_len=None if c["packed"] else c["T"])
    return {"dq": dq, "dk": dk, "dv": dv}


def _own_verify(s):
    import linear_attention_prefill_chunkwise_gb300 as lap
    lap.la_attn_verify(s["q"], s["k"], s["v"], s["case"]["D"] ** -0.5, s["k_cache"], s["v_cache"], s["cache_lens"],
                       s["case"]["T"], page_table=s["table"], mask=s["mask"], o=s["o"])
    return {"o": s["o"]}


def _own_commit(s):
    import linear_attention_prefill_chunkwise_gb300 as lap
    lap.la_attn_commit(s["k"], s["v"], s["k_cache"], s["v_cache"], s["cache_lens"],
                       T=None if s["case"]["prompt"] else s["case"]["T"], cu_seqlens=s["cu"],
                       accepted_len=s["accepted"], path=s["path"], page_table=s["table"])
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"]}


PLAIN = {"rope_fwd": _plain_rope, "rope_bwd": _plain_rope_bwd, "attn_fwd": _plain_attn, "attn_bwd": _plain_attn_bwd,
         "verify": _plain_verify, "commit": _plain_commit}
OWN = {"rope_fwd": _own_rope, "rope_bwd": _own_rope_bwd, "attn_fwd": _own_attn, "attn_bwd": _own_attn_bwd,
       "verify": _own_verify, "commit": _own_commit}


def run(state):
    return (OWN if own else PLAIN)[state["case"]["op"]](state)


# ------------------------------------------------------------------------------------------- work
def work(case):
    op, D, HK = case["op"], case["D"], case["HK"]
    if op in ("rope_fwd", "rope_bwd"):
        n, e = case["tokens"] * (case["H"] + HK) * D, 2 if case["dtype"] == "bf16" else 4
        small = 4 * case["tokens"] + 2 * case["R"] + 8 * D
        if op == "rope_fwd":
            return {"bytes": 2 * e * n + small, "flops": 8 * n}
        return {"bytes": 3 * e * n + small + 8 * D, "flops": 16 * n}
    if op in ("attn_fwd", "attn_bwd"):
        lens, H = _lengths(case), case["H"]
        n, products = sum(lens), H * sum(m * (m + 1) // 2 for m in lens)
        if op == "attn_fwd":
            return {"bytes": n * (4 * D * (H + HK) + 4 * H), "flops": 4 * D * products}
        return {"bytes": n * (8 * D * (H + HK) + 4 * H), "flops": 10 * D * products}
    lens = _cache_lengths(case)
    live = lens >= 0
    if op == "verify":
        B, T, H = int(live.sum()), case["T"], case["H"]
        keys = int(lens[live].sum())
        # a row of a tree sees few of the drafted tokens: the row itself counts here
        seen = T if case["tree"] else T * (T + 1) // 2
        return {"bytes": 4 * D * HK * (keys + B * T) + 4 * D * H * B * T,
                "flops": 4 * D * H * (T * keys + B * seen)}
    rows = int(_counts(case)[0][live].sum())
    return {"bytes": 8 * D * HK * rows, "flops": 0}


# ------------------------------------------------------------------------------------------ exact
def _exact_rope(s, x, w, inverse=False):
    """x normed (unless ``inverse``) and rotated as complex numbers, in 64 bits."""
    c = s["case"]
    R = c["R"]
    y = x if inverse else x / (x.pow(2).sum(-1, keepdim=True) / c["D"] + EPS).sqrt() * w.double()
    angle = torch.outer(s["pos"].double(), s["freq"].double())[:, None]
    unit = torch.polar(torch.ones_like(angle), -angle if inverse else angle)
    if c["pairs"] == "halves":
        z = torch.complex(y[..., : R // 2], y[..., R // 2:R]) * unit
        return torch.cat([z.real, z.imag, y[..., R:]], -1)
    z = torch.complex(y[..., 0:R:2], y[..., 1:R:2]) * unit
    return torch.cat([torch.view_as_real(z).flatten(-2), y[..., R:]], -1)


def _exact_attention(q, k, v, first, scale):
    """Row r of q [rows, D] sees keys 0 .. first + r: (o, lse) in 64 bits."""
    z = q @ k.T * scale
    keep = torch.arange(k.shape[0], device=q.device)[None] <= first + torch.arange(q.shape[0], device=q.device)[:, None]
    z = torch.where(keep, z, -math.inf)
    lse = torch.logsumexp(z, 1)
    return torch.exp(z - lse[:, None]), lse


def exact(case, seed):
    s = prepare(case, seed)
    op, D = case["op"], case["D"]
    if op == "rope_fwd":
        return {"q": _exact_rope(s, s["q"].double(), s["wq"]), "k": _exact_rope(s, s["k"].double(), s["wk"])}
    if op == "rope_bwd":
        out = {}
        for name, w in (("q", s["wq"]), ("k", s["wk"])):
            x, g = s[name].double(), _exact_rope(s, s[f"d{name}_out"].double(), None, inverse=True)
            ms = x.pow(2).sum(-1, keepdim=True) / D + EPS
            gw = g * w.double()
            out["d" + name] = gw / ms.sqrt() - x * (gw * x).sum(-1, keepdim=True) / (D * ms.pow(1.5))
            out["dw" + name] = (g * x / ms.sqrt()).sum((0, 1))
        return out
    scale = D ** -0.5
    if op in ("attn_fwd", "attn_bwd"):
        G, out = case["H"] // case["HK"], None
        q, k, v = (s[n].double() for n in ("q", "k", "v"))
        if op == "attn_fwd":
            out = {"o": torch.empty_like(q), "lse": torch.empty(s["q"].shape[:2][::-1], dtype=torch.float64, device=q.device)}
        else:
            out = {"dq": torch.empty_like(q), "dk": torch.zeros_like(k), "dv": torch.zeros_like(v)}
            do, delta = s["dout"].double(), (s["dout"].double() * s["o"].double()).sum(-1)
        lo = 0
        for n in s["lens"]:
            for h in range(case["H"]):
                for i in range(0, n, 2048):
                    j = min(n, i + 2048)
                    rows, keys = slice(lo + i, lo + j), slice(lo, lo + j)
                    kh, vh = k[keys, h // G], v[keys, h // G]
                    p, lse = _exact_attention(q[rows, h], kh, vh, i, scale)
                    if op == "attn_fwd":
                        out["o"][rows, h] = p @ vh
                        out["lse"][h, rows] = lse
                        continue
                    # the gradients' definition takes the stored lse and o as inputs
                    p = p * torch.exp(lse - s["lse"][h, rows].double())[:, None]
                    out["dv"][keys, h // G] += p.T @ do[rows, h]
                    ds = p * (do[rows, h] @ vh.T - delta[rows, h][:, None]) * scale
                    out["dq"][rows, h] = ds @ kh
                    out["dk"][keys, h // G] += ds.T @ q[rows, h]
            lo += n
        return out
    if op == "commit":
        return {"k_cache": _exact_commit(s, "k"), "v_cache": _exact_commit(s, "v")}
    T, H, HK = case["T"], case["H"], case["HK"]
    if int(np.maximum(s["lens"], 0).sum()) * T * H * D > 4e12:
        return None
    o = torch.zeros(s["o"].shape, dtype=torch.float64, device=s["o"].device)
    masks = None if s["mask"] is None else s["mask"].cpu().numpy().view(np.uint64)
    for b in range(case["B"]):
        n = int(s["lens"][b])
        if n < 0:
            continue
        seen = np.tril(np.ones((T, T), dtype=bool))
        if masks is not None:
            seen = np.array([[int(masks[b, t]) >> u & 1 for u in range(T)] for t in range(T)], dtype=bool)
        bias = torch.zeros((T, n + T), dtype=torch.float64, device=o.device)
        bias[:, n:][torch.from_numpy(~seen).to(o.device)] = -math.inf
        k, v = (torch.cat([_cached(s, x + "_cache", b, n), s[x][b * T:(b + 1) * T]]).double() for x in ("k", "v"))
        q = s["q"][b * T:(b + 1) * T].double().unflatten(1, (HK, H // HK))
        z = torch.einsum("thgd,nhd->hgtn", q, k) * scale + bias
        o[b * T:(b + 1) * T] = torch.einsum("hgtn,nhd->thgd", torch.softmax(z, -1), v).flatten(1, 2)
    return {"o": o}


def _exact_commit(s, name):
    """The cache after the writes, row by row."""
    case = s["case"]
    cache = s[name + "_cache"].double()
    counts, path = _counts(case)
    table = None if s["table"] is None else s["table"].cpu().numpy()
    size, x = cache.shape[1], s[name].double()
    first = np.concatenate([[0], np.cumsum(counts)]) if case["prompt"] else np.arange(case["B"]) * case["T"]
    for b in range(case["B"]):
        n = int(s["lens"][b])
        i = 0
        while n >= 0 and i < counts[b]:
            # a run of tokens that lie one after another in the cache
            at = n + i
            run_ = min(int(counts[b]) - i, size - at % size)
            rows = first[b] + np.arange(i, i + run_) if case["prompt"] else first[b] + path[b, i:i + run_]
            page = b if table is None else int(table[b, at // size])
            cache[page, at % size:at % size + run_] = x[torch.from_numpy(rows.astype(np.int64)).to(x.device)]
            i += run_
    return cache
