"""The long marked inputs themselves, without a GPU: every tile's loss is outside the tolerance."""
import numpy as np
import pytest

from attention_marked import QUERY, without_keys, tiles_of, tolerance, values_marked
from attention_reference import attend, causal


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
