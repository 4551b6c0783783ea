"""Which W4A4 shapes ask for a workspace, on the host: few rows whose K the weight
stream splits.  What the stream cannot split (one arrival counter for every group
of columns, 16384 of them; 65535 splits) runs as tiles, without a workspace."""
import os

import pytest

import block_scaled_precision_04_amd as bs
from block_scaled_precision_04_amd import _binding


@pytest.fixture(scope="module", autouse=True)
def blib():
    if not os.path.exists(_binding.LIB_PATH):
        from block_scaled_precision_04_amd import build
        build.build()


def _ws(M, N, K):
    return bs.workspace_bytes(bs.BS_OP_W4A4_MXFP4, M, N, K)


@pytest.mark.parametrize("M", [1, 8, 16])
def test_more_column_groups_than_counters(M):
    assert _ws(M, 48 * 16384, 5248) > 0            # 16384 groups of 48 columns
    assert _ws(M, 48 * 16384 + 16, 5248) == 0
    assert _ws(M, 800000, 5248) == 0


@pytest.mark.parametrize("M,steps", [(20, 8), (64, 8), (16, 40), (1, 40)])
def test_more_splits_than_a_grid_holds(M, steps):
    assert _ws(M, 16, 65535 * steps * 128) > 0     # runs of `steps` x 128 of K
    assert _ws(M, 16, (65535 * steps + 1) * 128) == 0


def test_rows_of_the_stream():
    assert _ws(16, 5120, 17408) > 0 and _ws(17, 8192, 17408) == 0
    assert _ws(64, 5120, 17408) > 0 and _ws(65, 5120, 17408) == 0 and _ws(64, 5120, 12160) == 0
