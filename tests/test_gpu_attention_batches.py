"""The bits of prompt attention and of its dq do not depend on what else is in the batch (GPU)."""
import numpy as np
import pytest

import linear_attention_prefill_chunkwise_gb300 as lap
from test_gpu_attention import make

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens,H,HK", [([700, 0, 1, 129, 300], 8, 2), ([2000, 128, 513], 5, 1), ([40] * 30 + [600], 4, 4)])
def test_a_sequence_alone_and_in_a_batch(lens, H, HK, D):
    rng = np.random.default_rng(sum(lens) + D)
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    q, k, v = make(rng, int(cu[-1]), (H, HK, HK), D, "fused")
    do, = make(rng, int(cu[-1]), (H,), D)
    dcu = torch.from_numpy(cu).cuda()
    o, lse = lap.la_attn_prefill_fwd(q, k, v, 0.15, cu_seqlens=dcu)
    dq = lap.la_attn_prefill_bwd(q, k, v, 0.15, o, lse, do, cu_seqlens=dcu)[0]
    for a, b in zip(cu, cu[1:]):
        if b > a:
            part = [t[a:b] for t in (q, k, v)]
            o1, lse1 = lap.la_attn_prefill_fwd(*part, 0.15, seq_len=int(b - a))
            dq1 = lap.la_attn_prefill_bwd(*part, 0.15, o1, lse1, do[a:b], seq_len=int(b - a))[0]
            assert torch.equal(o[a:b], o1) and torch.equal(lse[:, a:b], lse1) and torch.equal(dq[a:b], dq1)
