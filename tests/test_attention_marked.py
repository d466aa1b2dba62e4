"""The long marked inputs themselves, without a GPU: every tile's loss is outside the tolerance, and the pieces
for chosen rows and keys are those of the whole reference."""
import numpy as np
import pytest

from attention_marked import QUERY, keys_dkdv, prompt_marked, rows_dq, without_keys, tiles_of, tolerance, values_marked, weakest
from attention_reference import attend, attend_grad, causal


@pytest.mark.parametrize("D", [64, 128])
def test_a_lost_part_of_a_long_cache_shows(D):
    rng = np.random.default_rng(D)
    n, T = 20011, 3
    q, k, v = QUERY * rng.standard_normal((T, D)), rng.standard_normal((n + T, D)), values_marked(rng, n + T, D)
    seen = np.ones((T, n + T), bool)
    seen[:, n:] = causal(T, T)
    o, _, bound, _ = attend(q, k, v, seen, 0.15)
    # tiles, the last short one, and pages of 32
    for lost in tiles_of(n)[::9] + [slice(n // 128 * 128, n)] + [slice(i, i + 32) for i in range(0, n - 32, 1632)]:
        shown = np.abs(without_keys(q, k, v, seen, 0.15, lost) - o) / tolerance(o, bound)
        assert shown.max(1).min() > 2, (lost, shown.max(1))


@pytest.mark.parametrize("D,H,HK", [(64, 4, 2), (128, 2, 2)])
def test_a_lost_tile_of_a_long_prompts_gradients_shows(D, H, HK):
    rng = np.random.default_rng(D)
    T, heavy, rows = 2500, [0, 127, 128, 1300], [0, 127, 128, 1200, 2499]
    q, k, v, do, scale = prompt_marked(rng, T, H, HK, D, heavy)
    sums = {}
    for h in range(H):
        hk = h // (H // HK)
        o, lse, _, _ = attend(q[:, h], k[:, hk], v[:, hk], causal(T, T), scale)
        whole = attend_grad(q[:, h], k[:, hk], v[:, hk], scale, o, lse, do[:, h])
        dq = rows_dq(q[:, h], k[:, hk], v[:, hk], scale, o, lse, do[:, h], rows)
        np.testing.assert_allclose(dq[0], whole["dq"][0][rows], atol=1e-12)
        np.testing.assert_allclose(sum(dq[2]), dq[0], atol=1e-12)
        assert weakest(*dq, lambda r, i: rows[r] >= 128 and i <= rows[r] // 128) > 2
        for name, piece in keys_dkdv(q[:, h], k[:, hk], v[:, hk], scale, o, lse, do[:, h], heavy).items():
            np.testing.assert_allclose(piece[0], whole[name][0][heavy], atol=1e-11)
            a = sums.setdefault((hk, name), [0, 0, []])
            a[0], a[1], a[2] = a[0] + piece[0], a[1] + piece[1], a[2] + [(i, x) for i, x in enumerate(piece[2])]
    for (hk, name), (value, bound, shares) in sums.items():
        first = [i for i, _ in shares]
        assert weakest(value, bound, [x for _, x in shares], lambda r, i: first[i] >= heavy[r] // 128 + (name == "dk" and r == 0)) > 2, (hk, name)
