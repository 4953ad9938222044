"""The int8 GEMM plans' rules at their edges, without a GPU (host-only plans)."""
import pytest

import tile_scheduled_tensor_gb300 as tst


def _plan(M, N, K, **kw):
    return tst.gemm_int8_plan_create(M, N, K, host_only=True, **kw)


@pytest.mark.parametrize("num_sms", [1, 2, 3, 5])
@pytest.mark.parametrize("M,N,K,groups", [(200, 256, 512, 0), (97, 128, 16, 0), (8192, 8192, 1024, 0), (4000, 512, 2048, 3)])
def test_no_more_ctas_than_sms(M, N, K, groups, num_sms):
    p = _plan(M, N, K, groups=groups, num_sms=num_sms)
    assert p.info.tile_rows == 1 or 1 <= p.info.grid <= num_sms   # (1: no tiles)
    assert num_sms > 1 or p.info.tile_rows != 192                 # a pair takes two


@pytest.mark.parametrize("M,N", [(1000000, 200000), (65535 * 16, 2 ** 31 - 256), (65535 * 16, 1), (1, 2 ** 31 - 256)])
def test_the_form_without_tiles_has_no_limit_on_tiles(M, N):
    info = _plan(M, N, 16, num_sms=152, tile_rows=1).info
    assert (info.tile_rows, info.tile_cols, info.grid) == (1, 0, 0)


@pytest.mark.parametrize("rows,cols", [(16, 128), (32, 128), (64, 128), (128, 128), (192, 256)])
def test_tiles_up_to_their_limit(rows, cols):
    M = 2 ** 31 - 256
    tiles = -(-M // rows)
    most = (2 ** 30 - 1) // tiles   # columns of tiles
    if most * cols <= 2 ** 31 - 256:
        assert _plan(M, most * cols, 16, num_sms=152, tile_rows=rows).info.grid > 0
    if (most + 1) * cols <= 2 ** 31 - 256:
        with pytest.raises(tst.TstError) as e:
            _plan(M, most * cols + 1, 16, num_sms=152, tile_rows=rows)
        assert e.value.status == tst.TST_ERR_UNSUPPORTED
