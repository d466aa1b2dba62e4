"""The 8-bit values and scales of the RMS norm, bit by bit."""
import numpy as np
import pytest

import linear_attention_prefill_chunkwise_gb300 as lap

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def middles(top, count, seed):
    """FP32 values whose quotient by the scale of a group with maximum `top` is the middle between two e4m3
    numbers, but whose product with 448 / top is not."""
    top = np.float32(top)
    scale, inverse = top / np.float32(448), np.float32(448) / top
    rng = np.random.default_rng(seed)
    middle = ((rng.integers(8, 15, 20000) + 0.5) * np.exp2(rng.integers(-3, 5, 20000))).astype(np.float32)
    y = (middle * scale).astype(np.float32)
    y = y[(y / scale == middle) & (y * inverse != middle) & (y < top)]
    return y[:count]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("rows", [3, 1300])
def test_8_bit_values_and_scales_bit_by_bit(rows, group, dtype):
    """Rows of +-1 without eps have the norm 1, so y is the weight itself: scale is top / 448 and q is
    y (448 / top) rounded to the nearest e4m3, also where y / scale would be a tie."""
    C, tops = 4096, [3.3, 2.7, 4.9, 1.9] * 8 if group else [3.3]
    width = C // len(tops)
    y = np.concatenate([np.r_[np.float32(top), np.resize(middles(top, width - 1, k), width - 1)]
                        for k, top in enumerate(tops)])
    assert y.size == C and y.dtype == np.float32
    top = y[::width]
    sign = np.where(np.random.default_rng(1).random((rows, C)) < 0.5, -1, 1).astype(np.float32)
    x = torch.from_numpy(sign).to({"bf16": torch.bfloat16, "fp32": torch.float32}[dtype]).cuda()
    q, scales, _ = lap.la_rms_norm_fwd_fp8(x, torch.from_numpy(y).cuda(), 0.0, group=group)
    assert np.array_equal(scales.cpu().numpy(), np.tile(top / np.float32(448), (rows, 1)))
    # numpy's quotients are rounded divisions (a number over a torch tensor is a reciprocal and a product)
    want = torch.from_numpy((sign * y) * np.repeat(np.float32(448) / top, width))
    assert torch.equal(q.cpu().view(torch.uint8), want.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8))
