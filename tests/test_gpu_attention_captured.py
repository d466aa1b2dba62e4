"""A layer's calls captured into a graph while they take their workspaces themselves, replayed with new
values beside other work on the GPU."""
import numpy as np
import pytest

import linear_attention_prefill_chunkwise_gb300 as lap
from test_gpu_attention import make

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 128])
def test_workspaces_of_captured_calls(D):
    rng = np.random.default_rng(D)
    T, H, HK = 333, 8, 1
    q, k, v, do = make(rng, T, (H, HK, HK, H), D)
    w, pos = torch.ones(D, device="cuda"), torch.arange(T, dtype=torch.int32, device="cuda")
    freq = 10000.0 ** (-torch.arange(0, D, 2, device="cuda") / D)
    kc, vc = (t.view(64, 16, HK, D) for t in make(rng, 1024, (HK, HK), D))
    table = torch.arange(64, dtype=torch.int32, device="cuda")[None]
    held = torch.tensor([900], dtype=torch.int32, device="cuda")

    def layer():
        qr, kr = lap.la_qk_norm_rope_fwd(q, k, w, w, 1e-6, pos, freq)
        o, lse = lap.la_attn_prefill_fwd(qr, kr, v, D ** -0.5, seq_len=T)
        g = lap.la_attn_prefill_bwd(qr, kr, v, D ** -0.5, o, lse, do, seq_len=T)
        back = lap.la_qk_norm_rope_bwd(q, k, w, w, 1e-6, g[0], g[1], pos, freq)
        return qr, kr, o, lse, *g, *back, lap.la_attn_verify(qr[:4], kr[:4], v[:4], D ** -0.5, kc, vc, held, 4, page_table=table)
    layer()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = layer()
    for _ in range(3):
        q.copy_(torch.randn_like(q.float()))
        other = [torch.full((1 << n,), float("nan"), device="cuda") for n in (14, 16, 18, 20, 22)]
        graph.replay()
        ref = layer()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, ref))
        assert all(torch.isnan(t).all() for t in other)
