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
