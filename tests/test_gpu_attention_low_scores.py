"""Softmax attention on the GPU where a row's first keys, a whole tile of them, have scores below the
range of FP32 and later ones do not: they weigh nothing, whatever the scale."""
import numpy as np
import pytest

import linear_attention_prefill_chunkwise_gb300 as lap
from attention_reference import attend
from test_gpu_attention import check_backward, f64, make, near

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

LOW = 3e38  # times a query of 1000: beyond FP32


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("scale", [1.0, -0.75, 0.7, 0.125])
def test_prompt(scale, D):
    rng = np.random.default_rng(D)
    T, H, HK = 400, 4, 2
    q, k, v = make(rng, T, (H, HK, HK), D)
    q[:, :, 0], k[:, :, 0] = 1000.0, 0.0
    k[:128, :, 0] = -LOW if scale > 0 else LOW
    o, lse = lap.la_attn_prefill_fwd(q, k, v, scale, seq_len=T)
    for h in range(H):
        seen = np.arange(T)[None] <= np.arange(128, T)[:, None]
        ro, rl, eo, el = attend(f64(q[128:, h]), f64(k[:, h // 2]), f64(v[:, h // 2]), seen, scale)
        near(o[128:, h], ro, eo, f"o head {h}")
        near(lse[h, 128:], rl, el, f"lse head {h}", 2.0 ** -24)
    # rows from 128 on by themselves have the gradients that they have behind those keys
    do, = make(rng, T, (H,), D)
    dq, dk, dv = (g[128:] for g in lap.la_attn_prefill_bwd(q, k, v, scale, o, lse, do, seq_len=T))
    n = T - 128
    check_backward(q[128:], k[128:], v[128:], scale, [(0, n)], o[128:], lse[:, 128:], do[128:], (dq, dk, dv))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("scale", [1.0, 0.125])
@pytest.mark.parametrize("cached,low", [(300, 128), (3000, 2000), (3000, 3000)])
def test_drafted_tokens(cached, low, scale, D):
    """Also where a block's whole part of a request has such scores."""
    rng = np.random.default_rng(D + cached)
    T, H, HK = 3, 4, 1
    q, k, v = make(rng, T, (H, HK, HK), D)
    kc, vc = (t.unsqueeze(0) for t in make(rng, cached, (HK, HK), D))
    q[:, :, 0], k[:, :, 0], kc[..., 0] = 1000.0, 0.0, 0.0
    kc[:, :low, :, 0] = -LOW
    o = lap.la_attn_verify(q, k, v, scale, kc, vc, torch.tensor([cached], dtype=torch.int32, device="cuda"), T)
    keys, values = torch.cat([kc[0, :, 0], k[:, 0]]), torch.cat([vc[0, :, 0], v[:, 0]])
    seen = np.arange(cached + T)[None] <= cached + np.arange(T)[:, None]
    for h in range(H):
        ro, _, eo, _ = attend(f64(q[:, h]), f64(keys), f64(values), seen, scale)
        near(o[:, h], ro, eo, f"head {h}")
