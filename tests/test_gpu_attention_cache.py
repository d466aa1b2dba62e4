"""Drafted tokens over a key/value cache and the writes into it on the GPU (include/la_attention.h)
against the plain 64-bit form: paged and whole caches, tree masks, padded requests, foreign rows."""
import numpy as np
import pytest

import linear_attention_prefill_chunkwise_gb300 as lap
from attention_reference import BF16, attend, causal

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def f64(t):
    return t.detach().double().cpu().numpy()


def near(got, ref, bound, label):
    got = f64(got)
    assert np.all(np.isfinite(got)), f"{label}: non-finite"
    tol = bound + BF16 * (np.abs(ref) + bound) + 1e-30
    worst = np.max(np.abs(got - ref) / tol) if ref.size else 0.0
    assert worst <= 1, f"{label}: {worst:.3g} of its bound"


def bf(rng, *shape):
    return torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(torch.bfloat16).cuda()


def make_cache(rng, lens, HK, D, page, layout, fill=float("nan"), spare=3, width=None):
    """(k rows, v rows per request [len, HK, D], k_cache, v_cache, page_table); everything that holds no
    token is ``fill``."""
    B = len(lens)
    per = width or max(1, max(-(-max(n, 0) // page) for n in lens)) if page else 1
    pages, size = (B * per + spare, page) if page else (B + spare, max(1, max(lens)) + 5)
    if layout == "dense":
        kc, vc = (torch.full((pages, size, HK, D), fill, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    elif layout == "heads":  # head-major pages
        kc, vc = (torch.full((pages, HK, size, D), fill, dtype=torch.bfloat16, device="cuda").transpose(1, 2) for _ in range(2))
    elif layout == "pair":   # keys and values one after the other in a page
        both = torch.full((pages, 2, size, HK, D), fill, dtype=torch.bfloat16, device="cuda")
        kc, vc = both[:, 0], both[:, 1]
    else:                    # token by token
        both = torch.full((pages, size, 2, HK, D), fill, dtype=torch.bfloat16, device="cuda")
        kc, vc = both[:, :, 0], both[:, :, 1]
    table = torch.from_numpy(rng.permutation(pages)[:B * per].reshape(B, per).astype(np.int32)).cuda() if page else None
    ks, vs = [], []
    for b, n in enumerate(lens):
        n = max(n, 0)
        k, v = bf(rng, n, HK, D), bf(rng, n, HK, D)
        for i in range(0, n, size if page else max(n, 1)):
            pg = int(table[b, i // page]) if page else b
            m = min(n - i, size)
            kc[pg, :m], vc[pg, :m] = k[i:i + m], v[i:i + m]
        ks.append(k)
        vs.append(v)
        if page:  # behind the last page the table holds no page
            table[b, -(-n // page):] = -1
    return ks, vs, kc, vc, table


def random_tree(rng, B, T):
    bits = np.zeros((B, T), dtype=object)
    for b in range(B):
        for t in range(T):
            up = int(rng.integers(-1, t)) if t else -1
            bits[b, t] = (bits[b, up] if up >= 0 else 0) | 1 << t
    return bits


def to_int64(bits):
    return torch.from_numpy(np.vectorize(lambda x: int(x) - (1 << 64) if int(x) >= 1 << 63 else int(x), otypes=[np.int64])(bits)).cuda()


def check_verify(q, k, v, scale, ks, vs, lens, T, bits, o, before):
    H, HK = q.shape[1], k.shape[1]
    for b, n in enumerate(lens):
        rows = slice(b * T, (b + 1) * T)
        if n < 0:
            assert torch.equal(o[rows], before[rows])
            continue
        seen = np.ones((T, n + T), bool)
        seen[:, n:] = causal(T, T) if bits is None else [[int(bits[b, t]) >> u & 1 for u in range(T)] for t in range(T)]
        for h in range(H):
            hk = h // (H // HK)
            ref, _, bound, _ = attend(f64(q[rows, h]), np.concatenate([f64(ks[b][:, hk]), f64(k[rows, hk])]),
                                      np.concatenate([f64(vs[b][:, hk]), f64(v[rows, hk])]), seen, scale)
            near(o[rows, h], ref, bound, f"request {b} (length {n}) head {h}")


def run_verify(rng, lens, T, H, HK, D, page, layout="dense", tree=False, width=None, bits=None):
    B = len(lens)
    ks, vs, kc, vc, table = make_cache(rng, lens, HK, D, page, layout, width=width)
    q, k, v = bf(rng, B * T, H, D), bf(rng, B * T, HK, D), bf(rng, B * T, HK, D)
    if bits is None:
        bits = random_tree(rng, B, T) if tree else None
    o = torch.full((B * T, H, D), 7.0, dtype=torch.bfloat16, device="cuda")
    before = o.clone()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    dlens = torch.tensor(lens, dtype=torch.int32, device="cuda")
    ws = torch.full((lap.la_attn_verify_workspace(B, T, H, HK, D),), 255, dtype=torch.uint8, device="cuda")
    args = dict(page_table=table, mask=None if bits is None else to_int64(bits), dev_error=err)
    lap.la_attn_verify(q, k, v, 0.15, kc, vc, dlens, T, o=o, workspace=ws, **args)
    assert err.item() == 0
    check_verify(q, k, v, 0.15, ks, vs, lens, T, bits, o, before)
    again = before.clone()
    lap.la_attn_verify(q, k, v, 0.15, kc, vc, dlens, T, o=again, **args)
    assert torch.equal(o, again)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T", [1, 2, 5, 16, 33, 64])
@pytest.mark.parametrize("page", [0, 16, 48, 64, 128, 256])
def test_verify(page, T, D):
    rng = np.random.default_rng(page + T + D)
    lens = [0, 1, 130, -1, 127, 16, 300, 64, 257]
    for H, HK, layout in ((4, 2, "dense"), (3, 3, "heads")):
        run_verify(rng, lens, T, H, HK, D, page, layout)
    run_verify(rng, [40, 385], T, 5, 1, D, page, "pair", tree=True)
    run_verify(rng, [513], T, 2, 2, D, page, "tokens", tree=True)


@pytest.mark.parametrize("H,HK,T", [(8, 1, 1), (16, 1, 1), (64, 1, 3), (128, 1, 2), (40, 8, 7), (7, 1, 37), (24, 2, 64), (12, 12, 1)])
def test_grouped_heads(H, HK, T):
    rng = np.random.default_rng(H + T)
    run_verify(rng, [200, 0, 77], T, H, HK, 128, 32, tree=T > 1)
    run_verify(rng, [1000], T, H, HK, 64, 0)


@pytest.mark.parametrize("T", [65, 128, 129, 300])
def test_many_tokens_without_a_mask(T):
    rng = np.random.default_rng(T)
    run_verify(rng, [0, 100, 256, -1], T, 4, 2, 128, 64)
    run_verify(rng, [50], T, 3, 1, 64, 0)


@pytest.mark.parametrize("D", [64, 128])
def test_long_contexts_and_many_requests(D):
    rng = np.random.default_rng(D)
    run_verify(rng, [20011], 3, 4, 1, D, 64, width=400)        # one request over every SM
    run_verify(rng, [5000, 0, 12, 7777], 2, 8, 2, D, 16)
    run_verify(rng, [int(n) for n in rng.integers(-1, 40, 700)], 1, 2, 2, D, 16, width=9)
    run_verify(rng, [int(n) for n in rng.integers(-1, 3, 300)], 2, 2, 1, D, 0)


@pytest.mark.parametrize("D", [64, 128])
def test_rows_that_see_nothing(D):
    rng = np.random.default_rng(3)
    B, T = 4, 6
    bits = np.zeros((B, T), dtype=object)
    bits[1] = [1 << t for t in range(T)]
    bits[2, 3] = 0b100010
    bits[3, 5] = (1 << 63) | 1  # bits from T on are ignored
    run_verify(rng, [0, 0, 0, 0], T, 4, 2, D, 32, bits=bits)
    run_verify(rng, [130, 0, 0, 5], T, 4, 2, D, 32, bits=bits)
    run_verify(rng, [-1, -1, -1, -1], T, 4, 2, D, 32)


@pytest.mark.parametrize("D", [64, 128])
def test_non_finite_drafts_reach_only_rows_that_see_them(D):
    rng = np.random.default_rng(11)
    T, H, HK = 8, 4, 2
    ks, vs, kc, vc, table = make_cache(rng, [90, 20], HK, D, 16, "dense")
    q, k, v = bf(rng, 2 * T, H, D), bf(rng, 2 * T, HK, D), bf(rng, 2 * T, HK, D)
    bits = np.array([[1 << t | 1 for t in range(T)]] * 2, dtype=object)
    lens = torch.tensor([90, 20], dtype=torch.int32, device="cuda")
    args = dict(page_table=table, mask=to_int64(bits))
    clean = lap.la_attn_verify(q, k, v, 0.1, kc, vc, lens, T, **args)
    for bad in (float("nan"), float("inf")):
        k2, v2, q2 = k.clone(), v.clone(), q.clone()
        v2[5], k2[6], q2[7], v2[T + 3] = bad, bad, bad, bad
        got = lap.la_attn_verify(q2, k2, v2, 0.1, kc, vc, lens, T, **args)
        keep = [r for r in range(2 * T) if r not in (5, 6, 7, T + 3)]
        assert torch.equal(got[keep], clean[keep])
        assert not torch.isfinite(got[5]).all() and not torch.isfinite(got[T + 3]).all()


@pytest.mark.parametrize("D", [64, 128])
def test_non_finite_values_of_many_drafted_tokens(D):
    """Values that are not finite reach every later drafted token, also from the tiles of drafted tokens
    that a query tile sees whole, and no earlier one."""
    rng = np.random.default_rng(31)
    T, H, HK, n = 420, 8, 1, 70
    ks, vs, kc, vc, table = make_cache(rng, [n], HK, D, 16, "dense")
    q, k, v = bf(rng, T, H, D), bf(rng, T, HK, D), bf(rng, T, HK, D)
    v[5, 0, 3], v[131, 0, 40], v[300, 0, 7], v[419, 0, 0] = float("inf"), float("nan"), float("-inf"), float("inf")
    o = lap.la_attn_verify(q, k, v, 0.15, kc, vc, torch.tensor([n], dtype=torch.int32, device="cuda"), T, page_table=table)
    o = f64(o)
    for t, d, want in ((5, 3, np.inf), (131, 40, np.nan), (300, 7, -np.inf), (419, 0, np.inf)):
        assert np.isfinite(o[:t, :, d]).all()
        assert np.array_equal(o[t:, :, d], np.full((T - t, H), want), equal_nan=True)
    rest = np.ones(D, bool)
    rest[[3, 40, 7, 0]] = False
    assert np.isfinite(o[:, :, rest]).all()


def test_bad_lengths_and_pages_skip_their_request():
    rng = np.random.default_rng(12)
    D, T, H, HK, lens = 64, 2, 2, 1, [100, 60, 200, 30]
    ks, vs, kc, vc, table = make_cache(rng, lens, HK, D, 16, "dense", fill=0.0)
    q, k, v = bf(rng, 8, H, D), bf(rng, 8, HK, D), bf(rng, 8, HK, D)
    pages = kc.shape[0]
    for change, bit in ((("lens", 1, 16 * table.shape[1] + 1), lap.DEV_ERR_BAD_SEQLENS), (("lens", 1, 2 ** 31 - 1), lap.DEV_ERR_BAD_SEQLENS),
                        (("table", 1, pages), lap.DEV_ERR_BAD_INDEX), (("table", 1, -3), lap.DEV_ERR_BAD_INDEX),
                        (("table", 1, 2 ** 31 - 1), lap.DEV_ERR_BAD_INDEX)):
        dl, tb = torch.tensor(lens, dtype=torch.int32, device="cuda"), table.clone()
        if change[0] == "lens":
            dl[change[1]] = change[2]
        else:
            tb[change[1], 2] = change[2]
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        o = torch.full((8, H, D), 7.0, dtype=torch.bfloat16, device="cuda")
        before = o.clone()
        lap.la_attn_verify(q, k, v, 0.1, kc, vc, dl, T, page_table=tb, o=o, dev_error=err)
        assert err.item() == bit
        check_verify(q, k, v, 0.1, ks, vs, [100, -1, 200, 30], T, None, o, before)


def test_cache_past_32_bit_offsets():
    rng = np.random.default_rng(13)
    D, HK, page, T = 128, 2, 16, 2
    pages = (1 << 20) + 7  # 2^32 elements and more: 8.6 GB
    kc = torch.empty((pages, page, HK, D), dtype=torch.bfloat16, device="cuda")
    vc = torch.empty_like(kc)
    table = torch.tensor([[pages - 1, 0, pages // 2, pages - 3]], dtype=torch.int32, device="cuda")
    ks, vs = bf(rng, 60, HK, D), bf(rng, 60, HK, D)
    lens = torch.tensor([0], dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 60], dtype=torch.int32, device="cuda")
    lap.la_attn_commit(ks, vs, kc, vc, lens, cu_seqlens=cu, page_table=table)
    for i, p in enumerate(table[0].tolist()):
        n = min(16, 60 - 16 * i)
        assert torch.equal(kc[p, :n], ks[16 * i:16 * i + n]) and torch.equal(vc[p, :n], vs[16 * i:16 * i + n])
    q, k, v = bf(rng, T, 4, D), bf(rng, T, HK, D), bf(rng, T, HK, D)
    o = lap.la_attn_verify(q, k, v, 0.1, kc, vc, lens + 60, T, page_table=table)
    check_verify(q, k, v, 0.1, [ks], [vs], [60], T, None, o, o)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [0, 16, 64])
@pytest.mark.parametrize("layout", ["dense", "heads", "pair", "tokens"])
def test_commit(layout, page, D):
    rng = np.random.default_rng(page + D)
    lens, T, HK = [0, 13, -1, 64, 100, 31], 9, 3
    B = len(lens)
    room = [max(n, 0) + T + 40 for n in lens]
    _, _, kc, vc, table = make_cache(rng, room, HK, D, page, layout, fill=2.0)
    kc.fill_(2.0), vc.fill_(3.0)
    if page:
        assert int(table.min()) >= -1
    dl = torch.tensor(lens, dtype=torch.int32, device="cuda")

    def expect(rows):
        """The caches with token rows[b] = [source rows] written behind lens[b]."""
        a, c = torch.full_like(kc, 2.0), torch.full_like(vc, 3.0)
        for b, src in enumerate(rows):
            for i, r in enumerate(src):
                at = lens[b] + i
                pg, sl = (int(table[b, at // page]), at % page) if page else (b, at)
                a[pg, sl], c[pg, sl] = k[r], v[r]
        return a, c
    k, v = bf(rng, B * T, HK, D), bf(rng, B * T, 2 * HK, D)[:, HK:]
    acc = [4, 0, 5, 9, 20, -3]
    path = rng.integers(0, T, (B, T)).astype(np.int32)
    count = [min(max(a, 0), T) if n >= 0 else 0 for a, n in zip(acc, lens)]
    dacc, dpath = torch.tensor(acc, dtype=torch.int32, device="cuda"), torch.from_numpy(path).cuda()
    for over, rows in ((dict(accepted_len=dacc, path=dpath), [[b * T + int(path[b, i]) for i in range(count[b])] for b in range(B)]),
                       (dict(accepted_len=dacc), [[b * T + i for i in range(count[b])] for b in range(B)]),
                       (dict(), [[b * T + i for i in range(T)] if lens[b] >= 0 else [] for b in range(B)])):
        kc.fill_(2.0), vc.fill_(3.0)
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        lap.la_attn_commit(k, v, kc, vc, dl, T=T, page_table=table, dev_error=err, **over)
        a, c = expect(rows)
        assert torch.equal(kc, a) and torch.equal(vc, c) and err.item() == 0
    cuts = [0, 30, 30, 37, 38, 45, 54]
    kc.fill_(2.0), vc.fill_(3.0)
    lap.la_attn_commit(k, v, kc, vc, dl, cu_seqlens=torch.tensor(cuts, dtype=torch.int32, device="cuda"), page_table=table)
    a, c = expect([list(range(cuts[b], cuts[b + 1])) if lens[b] >= 0 else [] for b in range(B)])
    assert torch.equal(kc, a) and torch.equal(vc, c)


def test_commit_of_bad_requests_writes_the_others():
    rng = np.random.default_rng(14)
    D, HK, T, page = 64, 1, 4, 16
    k, v = bf(rng, 12, HK, D), bf(rng, 12, HK, D)
    table = torch.tensor([[0, 1], [2, 3], [4, 5]], dtype=torch.int32, device="cuda")
    good = torch.tensor([3, 14, 20], dtype=torch.int32, device="cuda")

    def run(lens=good, table=table, path=None, cu=None):
        kc, vc = (torch.zeros((6, page, HK, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        lap.la_attn_commit(k, v, kc, vc, lens, T=T if cu is None else None, cu_seqlens=cu, path=path, page_table=table, dev_error=err)
        return kc, err.item()
    want, err = run()
    assert err == 0

    def same_but(kc, pages):
        rest = [p for p in range(6) if p not in pages]
        return torch.equal(kc[rest], want[rest]) and not kc[pages].any()
    kc, err = run(lens=torch.tensor([3, 29, 20], dtype=torch.int32, device="cuda"))
    assert err == lap.DEV_ERR_BAD_SEQLENS and same_but(kc, [2, 3])
    tb = table.clone()
    tb[1, 1] = 6
    kc, err = run(table=tb)
    assert err == lap.DEV_ERR_BAD_INDEX and same_but(kc, [3])
    path = torch.arange(4, dtype=torch.int32, device="cuda").repeat(3, 1)
    path[2] = torch.tensor([0, 4, -1, 3])
    kc, err = run(path=path)
    assert err == lap.DEV_ERR_BAD_INDEX
    assert torch.equal(kc[5, 4], k[8]) and not kc[5, 5].any() and not kc[5, 6].any() and torch.equal(kc[5, 7], k[11])
    kc, err = run(cu=torch.tensor([0, 4, 3, 12], dtype=torch.int32, device="cuda"))
    assert err == lap.DEV_ERR_BAD_SEQLENS and torch.equal(kc[0], want[0]) and not kc[2:4].any()


def test_a_request_from_prompt_to_decode():
    """Prompt attention, commit, verify of a tree, commit of its path, decode: the outputs are those of
    one long prompt."""
    rng = np.random.default_rng(15)
    H, HK, D, page = 4, 2, 128, 16
    lens = [37, 150]
    total = [n + 4 for n in lens]  # three accepted drafts and one more token
    cu = np.concatenate([[0], np.cumsum(total)]).astype(np.int32)
    q, k, v = bf(rng, int(cu[-1]), H, D), bf(rng, int(cu[-1]), HK, D), bf(rng, int(cu[-1]), HK, D)
    whole, _ = lap.la_attn_prefill_fwd(q, k, v, 0.1, cu_seqlens=torch.from_numpy(cu).cuda())
    prompt = np.concatenate([np.arange(cu[b], cu[b] + lens[b]) for b in range(2)])
    pcu = torch.tensor([0, 37, 187], dtype=torch.int32, device="cuda")
    first, _ = lap.la_attn_prefill_fwd(q[prompt], k[prompt], v[prompt], 0.1, cu_seqlens=pcu)
    assert torch.equal(first, whole[prompt])
    kc, vc = (torch.full((24, page, HK, D), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    table = torch.from_numpy(rng.permutation(24)[:22].reshape(2, 11).astype(np.int32)).cuda()
    clens = torch.zeros(2, dtype=torch.int32, device="cuda")
    lap.la_attn_commit(k[prompt], v[prompt], kc, vc, clens, cu_seqlens=pcu, page_table=table)
    clens += torch.tensor(lens, dtype=torch.int32, device="cuda")
    # a tree of five drafts: 0 - 2 - 4 is the accepted path, 1 and 3 are others
    path, T = [0, 2, 4], 5
    dq, dk, dv = bf(rng, 2 * T, H, D), bf(rng, 2 * T, HK, D), bf(rng, 2 * T, HK, D)
    for b in range(2):
        for i, t in enumerate(path):
            r = int(cu[b]) + lens[b] + i
            dq[b * T + t], dk[b * T + t], dv[b * T + t] = q[r], k[r], v[r]
    mask = torch.tensor([[0b1, 0b11, 0b101, 0b1011, 0b10101]] * 2, device="cuda")
    o = lap.la_attn_verify(dq, dk, dv, 0.1, kc, vc, clens, T, page_table=table, mask=mask)
    ref = {b: f64(whole[cu[b]:cu[b + 1]]) for b in range(2)}
    for b in range(2):
        for i, t in enumerate(path):
            # both sides are within one rounding of P and of the output of the same value, of order 1
            assert np.abs(f64(o[b * T + t]) - ref[b][lens[b] + i]).max() <= 4 * BF16
    lap.la_attn_commit(dk, dv, kc, vc, clens, T=T, accepted_len=torch.tensor([3, 3], dtype=torch.int32, device="cuda"),
                       path=torch.tensor([path + [T, T]] * 2, dtype=torch.int32, device="cuda"), page_table=table)
    clens += 3
    last = np.array([int(cu[b + 1]) - 1 for b in range(2)])
    o = lap.la_attn_verify(q[last], k[last], v[last], 0.1, kc, vc, clens, 1, page_table=table)
    for b in range(2):
        assert np.abs(f64(o[b]) - ref[b][-1]).max() <= 4 * BF16


def test_captured_and_replayed_as_the_cache_grows():
    rng = np.random.default_rng(16)
    B, H, HK, D, page, T = 5, 8, 2, 64, 16, 2
    lens = [0, 50, 20, -1, 33]
    _, _, kc, vc, table = make_cache(rng, [n + 40 if n >= 0 else n for n in lens], HK, D, page, "dense")
    q, k, v = bf(rng, B * T, H, D), bf(rng, B * T, HK, D), bf(rng, B * T, HK, D)
    start = torch.tensor(lens, dtype=torch.int32, device="cuda")
    dl = start.clone()
    ws = torch.full((lap.la_attn_verify_workspace(B, T, H, HK, D),), 255, dtype=torch.uint8, device="cuda")
    o = torch.zeros((B * T, H, D), dtype=torch.bfloat16, device="cuda")

    def step():
        lap.la_attn_verify(q, k, v, 0.1, kc, vc, dl, T, page_table=table, o=o, workspace=ws)
        lap.la_attn_commit(k, v, kc, vc, dl, T=T, page_table=table)
        dl.add_((start >= 0).int() * T)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    dl.copy_(start)
    got = []
    for i in range(4):
        q.copy_(bf(np.random.default_rng(100 + i), B * T, H, D))
        graph.replay()
        got.append(o.clone())
    torch.cuda.synchronize()
    dl.copy_(start)
    for i in range(4):
        q.copy_(bf(np.random.default_rng(100 + i), B * T, H, D))
        step()
        assert torch.equal(o, got[i])


def test_a_page_table_without_columns_is_refused():
    """Its pointer is null, which is not to mean that requests have whole pages."""
    q = torch.zeros((4, 2, 64), dtype=torch.bfloat16, device="cuda")
    kc, vc = (torch.zeros((4, 16, 2, 64), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    lens, table = torch.zeros(4, dtype=torch.int32, device="cuda"), torch.zeros((4, 0), dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="column"):
        lap.la_attn_verify(q, q, q, 1.0, kc, vc, lens, 1, page_table=table)
    with pytest.raises(ValueError, match="column"):
        lap.la_attn_commit(q, q, kc, vc, lens, T=1, page_table=table)
    assert not kc.any() and not vc.any()


def test_wrong_arguments_are_refused():
    q = torch.zeros((4, 2, 64), dtype=torch.bfloat16, device="cuda")
    kc = torch.zeros((4, 16, 2, 64), dtype=torch.bfloat16, device="cuda")
    lens, table = torch.zeros(4, dtype=torch.int32, device="cuda"), torch.zeros((4, 1), dtype=torch.int32, device="cuda")
    for over, kind in ((dict(T=3), ValueError), (dict(T=0), ValueError), (dict(k_cache=kc[:, :, :1]), ValueError),
                       (dict(k_cache=kc.float()), TypeError), (dict(v_cache=kc[:2]), ValueError), (dict(cache_lens=lens[:3]), ValueError),
                       (dict(page_table=table[:3]), ValueError), (dict(page_table=table.long()), TypeError), (dict(cache_lens=None), TypeError),
                       (dict(mask=lens), TypeError), (dict(page_table=None, k_cache=kc[:2], v_cache=kc[:2]), lap.LaError),
                       (dict(workspace=torch.empty(1, dtype=torch.uint8, device="cuda")), lap.LaError)):
        a = dict(q=q, k=q, v=q, scale=1.0, k_cache=kc, v_cache=kc, cache_lens=lens, T=1, page_table=table)
        with pytest.raises(kind):
            lap.la_attn_verify(**{**a, **over})
    kc2 = torch.zeros_like(kc)
    for over, kind in ((dict(T=None), ValueError), (dict(cu_seqlens=lens), ValueError), (dict(T=3), ValueError),
                       (dict(path=lens), ValueError), (dict(v_cache=kc), lap.LaError), (dict(accepted_len=lens[:2]), ValueError)):
        a = dict(k=q, v=q, k_cache=kc, v_cache=kc2, cache_lens=lens, T=1, page_table=table)
        with pytest.raises(kind):
            lap.la_attn_commit(**{**a, **over})


def test_a_call_keeps_no_workspace():
    """The workspace that a call takes for itself is free again when it returns or raises, on any stream."""
    q = torch.zeros((4, 2, 64), dtype=torch.bfloat16, device="cuda")
    kc = torch.zeros((4, 16, 2, 64), dtype=torch.bfloat16, device="cuda")
    lens, o, side = torch.full((4,), 9, dtype=torch.int32, device="cuda"), torch.empty_like(q), torch.cuda.Stream()
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    for stream in (None, side, side.cuda_stream):
        lap.la_attn_verify(q, q, q, 0.1, kc, kc, lens, 1, o=o, stream=stream)
        assert torch.cuda.memory_allocated() == before
        torch.cuda.synchronize()
    with pytest.raises(lap.LaError):
        lap.la_attn_verify(q, q, q, float("nan"), kc, kc, lens, 1, o=o)
    assert torch.cuda.memory_allocated() == before
