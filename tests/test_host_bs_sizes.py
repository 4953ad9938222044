"""Sizes of block-scaled plans near 2^31 (host-only plans; no kernel runs).  The kernels count rows and
columns in 32 bits, and a tile's reach past the matrix: the first of a tile's 128 rows (256 columns) plus
127 (255) may not pass 2^31, or a row past the end would pass for one before it and be written."""
import pytest

import tile_scheduled_tensor_gb300 as tst

MOST = 2 ** 31 - 256


def _dense(M, N, **kw):
    # one column or row of tiles, so that listing the plan's work stays short
    return tst.gemm_plan_create(M, N, 16, dtype="e4m3", schedule="persistent", host_only=True, num_sms=152, **kw)


def _grouped(M, N, groups=2, **kw):
    return tst.gemm_grouped_plan_create(groups, M, N, 16, dtype="e4m3", host_only=True, num_sms=152, **kw)


@pytest.mark.parametrize("ab", [(1, 128, 128), (1, 128, 1), (1, 32), (128, 128)])
def test_block_scaled_plans_end_below_two_to_the_31(ab):
    for over in (2 ** 31 - 1, MOST + 1):
        for make, M, N in ((_dense, over, 8), (_dense, 8, over), (_grouped, over, 8), (lambda M, N, **kw: _grouped(M, N, 1, **kw), 8, over)):
            with pytest.raises(tst.TstError) as e:
                make(M, N, ab_block=ab)
            assert e.value.status == tst.TST_ERR_UNSUPPORTED, (M, N)


@pytest.mark.parametrize("ab", [(1, 128, 128), (1, 128, 1)])
def test_the_largest_size_is_taken(ab):
    info = _grouped(MOST, 8, ab_block=ab).info
    # rows and columns that a tile may name, in 32 bits: a group may start anywhere up to the last row
    assert MOST + info.bm - 1 < 2 ** 31 and MOST + info.bn - 1 < 2 ** 31
    assert _grouped(8, MOST, 1, ab_block=ab).info.bn in (128, 256)


def test_other_plans_keep_their_sizes():
    assert _grouped(2 ** 31 - 1, 8).info.bm in (128, 256)
