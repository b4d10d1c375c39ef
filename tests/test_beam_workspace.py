"""What the merge of the selection takes into shared memory, seen from the workspace's size (CPU only)."""

import pytest


@pytest.fixture(scope="module")
def kv():
    from calibration_free_kv_gb300 import build
    build.build()
    from calibration_free_kv_gb300 import kvarn
    return kvarn


@pytest.mark.parametrize("beams", [1, 2, 3, 5, 8, 16, 17, 31, 32])
@pytest.mark.parametrize("count", [1, 2, 7, 16, 33, 63, 64])
@pytest.mark.parametrize("vocab", [1, 2049, 50_257, 1 << 20, 1 << 26])
def test_candidates_of_a_group(kv, vocab, count, beams):
    # A group's lists: 8 bytes a chunk for its sum, 8 a candidate.  The merge takes 12 bytes a candidate without a raised
    # limit, 2048 at most; rows are divided only up to 1024.
    most = max(1024, beams * count)
    assert most <= 2048
    for batch in (1, 7, 400):
        size = kv.beam_select_workspace_bytes(batch, beams, vocab, count)
        assert 0 < size <= batch * (most * 8 + most * 8 // count) + 32
