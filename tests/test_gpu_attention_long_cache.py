"""Drafted tokens over long caches on the GPU, over values in which every tile of keys counts (attention_marked)."""
import numpy as np
import pytest

import linear_attention_prefill_chunkwise_gb300 as lap
from attention_marked import QUERY, without_keys, tiles_of, tolerance, values_marked
from attention_reference import attend, causal
from test_gpu_attention import f64, near

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def bf(x):
    return torch.from_numpy(np.asarray(x, dtype=np.float32)).to(torch.bfloat16).cuda()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens,T,H,HK,page,tree", [
    ([20011], 3, 4, 1, 64, False),              # one request over every SM
    ([20011], 1, 2, 2, 0, False),
    ([5000, 0, 12, 7777], 2, 8, 2, 16, False),
    ([9000], 40, 8, 1, 32, True),               # query tiles of 16 tokens
    ([3000, 6001], 150, 2, 1, 48, False)])      # tiles of drafted tokens too
def test_every_tile_of_a_long_cache(lens, T, H, HK, page, tree, D):
    rng = np.random.default_rng(sum(lens) + T + D)
    B, size = len(lens), page or max(lens) + 3
    per = -(-max(lens) // size)
    pages = B * per + 2
    kc, vc = (torch.full((pages, size, HK, D), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    table = rng.permutation(pages)[:B * per].reshape(B, per) if page else np.arange(B)[:, None]
    q, k, v = bf(QUERY * rng.standard_normal((B * T, H, D))), bf(rng.standard_normal((B * T, HK, D))), torch.empty((B * T, HK, D), dtype=torch.bfloat16, device="cuda")
    keys, values = [], []
    for b, n in enumerate(lens):
        ks = bf(rng.standard_normal((n, HK, D)))
        vs = bf(np.stack([values_marked(rng, n + T, D) for _ in range(HK)], 1))
        at = torch.from_numpy(table[b][np.arange(n) // size] * size + np.arange(n) % size).cuda()
        kc.view(-1, HK, D)[at], vc.view(-1, HK, D)[at], v[b * T:(b + 1) * T] = ks, vs[:n], vs[n:]
        keys.append(f64(torch.cat([ks, k[b * T:(b + 1) * T]])))
        values.append(f64(vs))
    # every other drafted token starts a branch of its own behind the first
    bits = [1 | 1 << t | (1 << t - 1 if t % 2 == 0 and t else 0) for t in range(T)] if tree else None
    among = np.array([[m >> u & 1 for u in range(T)] for m in bits], bool) if tree else causal(T, T)
    mask = torch.tensor([bits] * B, device="cuda") if tree else None
    o = lap.la_attn_verify(q, k, v, 0.15, kc, vc, torch.tensor(lens, dtype=torch.int32, device="cuda"), T, mask=mask,
                           page_table=torch.from_numpy(table.astype(np.int32)).cuda() if page else None)
    for b, n in enumerate(lens):
        seen = np.ones((T, n + T), bool)
        seen[:, n:] = among
        for h in range(H):
            rows, hk = slice(b * T, (b + 1) * T), h // (H // HK)
            ref, _, bound, _ = attend(f64(q[rows, h]), keys[b][:, hk], values[b][:, hk], seen, 0.15)
            near(o[rows, h], ref, bound, f"request {b} (length {n}) head {h}")
            for lost in tiles_of(n)[::17] if h == 0 and n > 128 else []:
                less = without_keys(f64(q[rows, h]), keys[b][:, hk], values[b][:, hk], seen, 0.15, lost)
                assert (np.abs(less - ref) / tolerance(ref, bound)).max(1).min() > 2, lost
