"""The gated recurrence's host side at its limits, without a GPU."""
import pytest

import linear_attention_prefill_chunkwise_gb300 as lap

torch = pytest.importorskip("torch")
UNSUPPORTED = 2


@pytest.mark.parametrize("T", [13, 25, 26])
def test_tiles_times_columns_stay_below_two_to_the_thirty(T):
    """FP32 gradients of unaligned rows have tiles of 24 rows, and sequences of 13 to 26 tokens fill little
    more than half of theirs: a batch whose tiles would pass 2^30 is refused, by any rows per tile."""
    tiles = -(-T // 24)
    columns = 8
    most = (1 << 30) // (tiles * columns)  # sequences
    with pytest.raises(lap.LaError) as e:
        lap.la_gated_scan_workspace(most + 1, T, most + 1, 64 * columns, False, torch.float32, True)
    assert e.value.status == UNSUPPORTED
    assert lap.la_gated_scan_workspace(most // 3, T, most // 3, 64 * columns, False, torch.float32, True) > 0


@pytest.mark.parametrize("t,stride", [(torch.zeros(1, 8).t(), 1), (torch.zeros(3, 8).t()[:, 1:2], 1),
                                      (torch.zeros(8, 5)[:, 2:3], 5), (torch.zeros(8, 2, 3)[:, :, 1][:, :1], 6),
                                      (torch.zeros(6).expand(1, 6), 6), (torch.zeros(0, 4), 4)])
def test_row_strides_of_single_columns_and_rows(t, stride):
    """A single column may have any column stride."""
    assert lap._stride(t, "x", *t.shape) == stride


@pytest.mark.parametrize("t", [torch.zeros(8, 1).expand(8, 4), torch.zeros(1).expand(8, 1), torch.zeros(4, 8).t(),
                               torch.zeros(8).expand(4, 8)])
def test_other_strides_are_refused(t):
    with pytest.raises(ValueError, match="x"):
        lap._stride(t, "x", *t.shape)


@pytest.mark.parametrize("dtype", [torch.float16, torch.float64, "bf16", None])
def test_workspace_of_an_unknown_type_is_refused(dtype):
    with pytest.raises(TypeError, match="bfloat16 or torch.float32"):
        lap.la_gated_scan_workspace(1, 600, 3, 64, True, dtype, True)
