"""Scales that the attention calls refuse, without a GPU: what is not finite, or not once the kernels
have multiplied it by log2 e (every score would then be infinite or 0 * inf)."""
import pytest

from test_attention import INVALID, attn, attn_back, verify


@pytest.mark.parametrize("call", [attn, attn_back, verify])
@pytest.mark.parametrize("scale", [2.5e38, -2.5e38, 3e38, float("inf"), -float("inf"), float("nan")])
def test_scales_without_a_meaning_are_refused(call, scale):
    assert call(scale=scale) == INVALID


@pytest.mark.parametrize("call", [attn, attn_back, verify])
@pytest.mark.parametrize("scale", [0.0, -1.0, 1e-38, 1.9e38, -1.9e38])
def test_other_scales_are_not(call, scale):
    torch = pytest.importorskip("torch")
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")  # (the buffers are fake: past the host checks the device query fails)
    assert call(scale=scale) != INVALID
