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
