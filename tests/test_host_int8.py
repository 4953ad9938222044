"""The int8 GEMM calls without a GPU: plan rules and refusals at the C boundary (host-only plans; no
kernel runs)."""
import ctypes

import pytest

import tile_scheduled_tensor_gb300 as tst
from tile_scheduled_tensor_gb300 import _capi


def _plan(M=100, N=256, K=512, **kw):
    return tst.gemm_int8_plan_create(M, N, K, **dict(dict(host_only=True, num_sms=152), **kw))


def test_plan_rules_and_info():
    p = _plan(groups=4, tile_rows=16)
    assert (p.info.M, p.info.N, p.info.K, p.info.groups) == (100, 256, 512, 4)
    assert p.info.tile_cols >= 128 and p.info.grid >= 1 and 0 < p.info.smem_bytes <= 232448
    invalid, align, unsupported = tst.TST_ERR_INVALID_ARG, tst.TST_ERR_ALIGNMENT, tst.TST_ERR_UNSUPPORTED
    for kw, status in ((dict(M=0), invalid), (dict(N=0), invalid), (dict(K=0), invalid), (dict(M=1 << 31), invalid), (dict(groups=-1), invalid),
                       (dict(out_dtype="e4m3"), invalid), (dict(out_dtype=9), invalid), (dict(num_sms=0), invalid), (dict(num_sms=-1), invalid),
                       (dict(timeout_ns=-1), invalid), (dict(tile_rows=-1), invalid), (dict(tile_rows=48), unsupported),
                       (dict(tile_rows=1, M=(1 << 20) + 1), unsupported), (dict(tile_rows=1, M=65535 * 16 + 1), unsupported),
                       (dict(tile_rows=192, num_sms=1), unsupported), (dict(K=520), align), (dict(K=131072), unsupported), (dict(groups=513), unsupported),
                       (dict(M=(1 << 31) - 255), unsupported), (dict(N=1 << 23, groups=256), unsupported)):
        with pytest.raises(tst.TstError) as e:
            _plan(**kw)
        assert e.value.status == status, kw
    _plan(K=131056), _plan(groups=512), _plan(tile_rows=1, M=65535 * 16)
    for rows in (1, 16, 32, 64, 128, 192):
        assert _plan(tile_rows=rows).info.tile_rows == rows
    assert _plan(M=16384, N=4096).info.workspace_bytes >= 2 * 16384 * 512 > _plan(M=8).info.workspace_bytes   # A in FP16
    assert tst.lib.gemm_int8_plan_create(None, 1, 1, 16, None) == invalid
    h = ctypes.c_void_p(1)
    assert tst.lib.gemm_int8_plan_create(ctypes.byref(h), 1, 1, 16, None) == invalid and not h.value
    assert tst.lib.gemm_int8_plan_destroy(None) == tst.TST_OK
    assert tst.lib.gemm_int8_plan_get_info(None, ctypes.byref(_capi.tst_int8_plan_info())) == invalid
    assert tst.lib.gemm_int8_status_query(None) == invalid and tst.lib.gemm_int8_status_query(p._h) == tst.TST_ERR_NO_DEVICE
    tst.gemm_int8_plan_destroy(p)
    tst.gemm_int8_plan_destroy(p)
    with pytest.raises(ValueError):
        p._h


# addresses that are only checked, never read: a host-only plan stops before any launch
A16, A8, A4, A2 = 1 << 20, (1 << 20) + 8, (1 << 20) + 4, (1 << 20) + 2


def test_run_refusals():
    dense, grouped = _plan(), _plan(groups=4, out_dtype="f32", has_bias=True)
    good = dict(plan=dense._h, group_rows=None, A=A16, B=A16, D=A2, row_scale=A4, col_scale=A4, bias=None, stream=None)

    def call(**kw):
        return tst.lib.gemm_int8_run(*dict(good, **kw).values())
    mine = dict(plan=grouped._h, group_rows=A4, D=A4, bias=A4)
    assert call() == tst.TST_ERR_NO_DEVICE and call(bias=A2 + 1) == tst.TST_ERR_NO_DEVICE   # an unused bias is ignored
    assert call(**mine) == tst.TST_ERR_NO_DEVICE
    for kw in (dict(plan=None), dict(A=None), dict(B=None), dict(D=None), dict(row_scale=None), dict(col_scale=None), dict(group_rows=A4),
               dict(mine, group_rows=None), dict(mine, bias=None)):
        assert call(**kw) == tst.TST_ERR_INVALID_ARG, kw
    for kw in (dict(A=A8), dict(B=A8), dict(D=A2 + 1), dict(row_scale=A2), dict(col_scale=A2), dict(mine, D=A2), dict(mine, group_rows=A2),
               dict(mine, bias=A2)):
        assert call(**kw) == tst.TST_ERR_ALIGNMENT, kw
