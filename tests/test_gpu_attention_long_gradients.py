"""Gradients of long prompts on the GPU, over inputs in which every tile of keys, and of rows of every head,
counts (attention_marked)."""
import numpy as np
import pytest

import linear_attention_prefill_chunkwise_gb300 as lap
from attention_marked import keys_dkdv, prompt_marked, rows_dq, weakest
from attention_reference import attend
from test_gpu_attention import f64, near

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def bf(x):
    return torch.from_numpy(np.asarray(x, dtype=np.float32)).to(torch.bfloat16).cuda()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T,H,HK", [(9001, 4, 2),     # heads of a group in parts
                                    (9001, 10, 5),    # more items than SMs, whole groups
                                    (5100, 7, 7)])
def test_every_tile_of_a_long_prompts_gradients(T, H, HK, D):
    rng = np.random.default_rng(T + H + D)
    heavy, rows = [0, 1, 127, 128, 4000, T - 300], [0, 127, 128, 255, 4200, T - 500, T - 1]
    *given, scale = prompt_marked(rng, T, H, HK, D, heavy)
    q, k, v, do = (bf(x) for x in given)
    o, lse = lap.la_attn_prefill_fwd(q, k, v, scale, seq_len=T)
    dq, dk, dv = lap.la_attn_prefill_bwd(q, k, v, scale, o, lse, do, seq_len=T)
    Q, K, V, O, L, DO = (f64(t) for t in (q, k, v, o, lse, do))
    sums = {}
    for h in range(H):
        hk = h // (H // HK)
        one = (Q[:, h], K[:, hk], V[:, hk], scale, O[:, h], L[h], DO[:, h])
        r = [0, 128, 4096, T - 1]
        seen = np.arange(T)[None] <= np.array(r)[:, None]
        ro, rl, eo, el = attend(Q[r, h], K[:, hk], V[:, hk], seen, scale)
        near(o[r, h], ro, eo, f"o head {h}")
        near(lse[h, r], rl, el, f"lse head {h}", 2.0 ** -24)
        value, bound, shares = rows_dq(*one, rows)
        near(dq[rows, h], value, bound, f"dq head {h}")
        assert weakest(value, bound, shares, lambda r, i: rows[r] >= 128 and i <= rows[r] // 128) > 2
        for name, piece in keys_dkdv(*one, heavy).items():
            a = sums.setdefault((hk, name), [0, 0, []])
            a[0], a[1], a[2] = a[0] + piece[0], a[1] + piece[1], a[2] + list(enumerate(piece[2]))
    for (hk, name), (value, bound, shares) in sums.items():
        near((dk if name == "dk" else dv)[heavy, hk], value, bound, f"{name} head {hk}")
        tile = [i for i, _ in shares]
        # (tile 0 holds few rows that see two heavy keys, whose dS is near zero)
        assert weakest(value, bound, [x for _, x in shares], lambda r, i: tile[i] >= max(1, heavy[r] // 128)) > 2, (hk, name)
