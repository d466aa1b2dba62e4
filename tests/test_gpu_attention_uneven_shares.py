"""Prompt gradients on the GPU whose shares of a group's heads are not even."""
import numpy as np
import pytest

import linear_attention_prefill_chunkwise_gb300 as lap
from test_gpu_attention import check_backward, make

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens,H,HK,parts", [
    ([700], 40, 8, 3),                 # 5 heads in 2, 2 and 1
    ([300, 500], 40, 8, 2),            # 3 and 2
    ([129, 400, 1000], 14, 2, 4),      # 7 in 2, 2, 2 and 1
    ([1500, 1, 900], 14, 2, 4),        # of the 7 parts that the workspace has room for
    ([1500, 1, 900], 11, 1, 6)])       # of 11
def test_uneven_shares_of_a_groups_heads(lens, H, HK, parts, D):
    """The parts are seen in the workspace, which holds NaN before: sums in ``parts`` planes and no more, of the
    sequences' rows alone."""
    rng = np.random.default_rng(sum(lens) + H)
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    tokens = int(cu[-1]) + 30
    q, k, v = make(rng, tokens, (H, HK, HK), D, "fused")
    do, = make(rng, tokens, (H,), D)
    dcu = torch.from_numpy(cu).cuda()
    o, lse = lap.la_attn_prefill_fwd(q, k, v, 0.15, cu_seqlens=dcu)
    ws = torch.full((lap.la_attn_prefill_bwd_workspace(1, tokens, H, HK, D),), 255, dtype=torch.uint8, device="cuda")
    grads = [torch.full((tokens, n, D), 7.0, dtype=torch.bfloat16, device="cuda") for n in (H, HK, HK)]
    lap.la_attn_prefill_bwd(q, k, v, 0.15, o, lse, do, cu_seqlens=dcu, dq=grads[0], dk=grads[1], dv=grads[2], workspace=ws)
    check_backward(q, k, v, 0.15, [(a, b) for a, b in zip(cu, cu[1:]) if b > a], o, lse, do, grads)
    assert all((g[cu[-1]:] == 7).all() for g in grads)
    sums = ws[-(-4 * H * tokens // 256) * 256:]  # behind delta
    plane = 2 * HK * tokens * D
    planes = sums[:4 * plane * parts].view(torch.float32).view(parts, 2, HK, tokens, D)
    assert torch.isfinite(planes[:, :, :, :cu[-1]]).all() and torch.isnan(planes[:, :, :, cu[-1]:]).all()
    marks = -(-4 * plane * parts // 256) * 256
    assert (sums[marks:marks + HK * tokens].view(HK, tokens) == torch.arange(tokens, device="cuda").lt(int(cu[-1])).byte()).all()
    assert (sums[marks + -(-HK * tokens // 256) * 256:] == 255).all()
