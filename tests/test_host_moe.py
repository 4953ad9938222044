"""The mixture-of-experts calls without a GPU: plan rules, refusals at the C boundary, and grouped
block-scaled plans (host-only plans; no kernel runs)."""
import ctypes

import pytest

import tile_scheduled_tensor_gb300 as tst
from tile_scheduled_tensor_gb300 import _capi


def _plan(T=100, E=64, k=8, **kw):
    return tst.moe_plan_create(T, E, k, host_only=True, **kw)


def test_plan_rules_and_info():
    info = tst.moe_plan_get_info(_plan(normalize=False, balance_coef=0.5))
    assert (info.max_tokens, info.experts, info.top_k, info.normalize, info.balance_coef) == (100, 64, 8, 0, 0.5)
    # 8 bytes per expert and chunk of 32 tokens (65 rows of counts), and two small blocks
    assert info.workspace_bytes == 256 + 256 + 2 * 1280
    for T, E, k, status in ((0, 8, 2, tst.TST_ERR_INVALID_ARG), (4, 0, 1, tst.TST_ERR_INVALID_ARG),
                            (4, 8, 0, tst.TST_ERR_INVALID_ARG), (4, 8, 9, tst.TST_ERR_INVALID_ARG),
                            (1 << 30, 8, 2, tst.TST_ERR_INVALID_ARG), (4, 1025, 2, tst.TST_ERR_UNSUPPORTED),
                            (4, 64, 33, tst.TST_ERR_UNSUPPORTED)):
        with pytest.raises(tst.TstError) as e:
            _plan(T, E, k)
        assert e.value.status == status, (T, E, k)
    with pytest.raises(tst.TstError) as e:
        _plan(balance_coef=float("nan"))
    assert e.value.status == tst.TST_ERR_INVALID_ARG
    assert tst.lib.moe_plan_create(None, 4, 8, 2, None) == tst.TST_ERR_INVALID_ARG
    h = ctypes.c_void_p(1)
    assert tst.lib.moe_plan_create(ctypes.byref(h), 4, 8, 2, None) == tst.TST_ERR_INVALID_ARG and not h.value
    assert tst.lib.moe_plan_destroy(None) == tst.TST_OK
    assert tst.lib.moe_plan_get_info(None, ctypes.byref(_capi.tst_moe_plan_info())) == tst.TST_ERR_INVALID_ARG
    assert tst.lib.moe_status_query(None) == tst.TST_ERR_INVALID_ARG


def test_destroyed_plan_is_refused():
    p = _plan()
    tst.moe_plan_destroy(p)
    tst.moe_plan_destroy(p)
    with pytest.raises(ValueError):
        tst.moe_plan_get_info(p)


# addresses that are only checked, never read: a host-only plan stops before any launch
A16, A8, A4, A2 = 1 << 20, (1 << 20) + 8, (1 << 20) + 4, (1 << 20) + 2
F32, BF16, E4M3 = tst.TST_OUT_F32, tst.TST_OUT_BF16, tst.TST_OUT_E4M3


def test_route_refusals():
    p = _plan()
    good = dict(plan=p._h, tokens=10, logits=A16, dtype=F32, ld=64, mask=None, expert=A4, weight=A4, row=A4, counts=A4,
                totals=A4, loss=A4, stream=None)

    def call(**kw):
        return tst.lib.moe_route(*dict(good, **kw).values())
    assert call() == tst.TST_ERR_NO_DEVICE and call(tokens=0, logits=None, expert=None) == tst.TST_ERR_NO_DEVICE
    for kw in (dict(plan=None), dict(tokens=-1), dict(tokens=101), dict(dtype=E4M3), dict(dtype=7), dict(ld=63),
               dict(logits=None), dict(expert=None), dict(weight=None), dict(row=None), dict(counts=None), dict(totals=None),
               dict(loss=None)):
        assert call(**kw) == tst.TST_ERR_INVALID_ARG, kw
    for kw in (dict(logits=A2), dict(dtype=BF16, logits=A2 + 1), dict(expert=A2), dict(loss=A2)):
        assert call(**kw) == tst.TST_ERR_ALIGNMENT, kw
    grad = dict(plan=p._h, tokens=10, logits=A16, dtype=F32, ld=64, mask=None, expert=A4, counts=A4, totals=A4, d_weight=None,
                d_loss=None, d_logits=A16, d_ld=64, stream=None)
    back = lambda **kw: tst.lib.moe_route_backward(*dict(grad, **kw).values())  # noqa: E731
    assert back() == tst.TST_ERR_NO_DEVICE
    for kw in (dict(d_ld=63), dict(d_logits=None), dict(expert=None), dict(counts=None), dict(totals=None), dict(tokens=101)):
        assert back(**kw) == tst.TST_ERR_INVALID_ARG, kw
    assert back(d_logits=A2) == tst.TST_ERR_ALIGNMENT and back(d_loss=A2) == tst.TST_ERR_ALIGNMENT


def test_row_refusals():
    p = _plan()
    disp = dict(plan=p._h, tokens=10, hidden=64, x=A16, x_dtype=BF16, x_ld=64, row=A4, rows=A16, rows_dtype=E4M3, n_rows=80,
                scales=A4, stream=None)
    d = lambda **kw: tst.lib.moe_dispatch(*dict(disp, **kw).values())  # noqa: E731
    assert d() == tst.TST_ERR_NO_DEVICE and d(row=None) == tst.TST_ERR_NO_DEVICE
    assert d(row=None, tokens=800, n_rows=800) == tst.TST_ERR_NO_DEVICE   # rows in order: up to tokens x top_k
    for kw in (dict(hidden=0), dict(x_ld=63), dict(x_dtype=E4M3), dict(rows_dtype=5), dict(x=None), dict(rows=None),
               dict(scales=None), dict(n_rows=-1), dict(tokens=101), dict(row=None, n_rows=9), dict(row=None, tokens=801)):
        assert d(**kw) == tst.TST_ERR_INVALID_ARG, kw
    for kw in (dict(hidden=72, x_ld=72), dict(rows=A8), dict(x=A16 + 1), dict(scales=A2)):
        assert d(**kw) == tst.TST_ERR_ALIGNMENT, kw
    assert d(rows_dtype=F32) == tst.TST_ERR_UNSUPPORTED
    assert d(rows_dtype=BF16, scales=None, hidden=63) == tst.TST_ERR_NO_DEVICE
    comb = dict(plan=p._h, tokens=10, hidden=63, rows=A16, rows_dtype=BF16, n_rows=80, row=A4, weight=None, out=A4,
                out_dtype=F32, out_ld=63, stream=None)
    c = lambda **kw: tst.lib.moe_combine(*dict(comb, **kw).values())  # noqa: E731
    assert c() == tst.TST_ERR_NO_DEVICE and c(n_rows=0, rows=None) == tst.TST_ERR_NO_DEVICE
    for kw in (dict(rows=None), dict(row=None), dict(out=None), dict(out_ld=62), dict(rows_dtype=E4M3), dict(out_dtype=E4M3)):
        assert c(**kw) == tst.TST_ERR_INVALID_ARG, kw
    assert c(out=A2) == tst.TST_ERR_ALIGNMENT
    back = dict(plan=p._h, tokens=10, hidden=63, rows=A16, rows_dtype=BF16, n_rows=80, row=A4, weight=A4, d_out=A4, out_dtype=F32,
                d_out_ld=63, d_rows=A16, d_weight=A4, stream=None)
    b = lambda **kw: tst.lib.moe_combine_backward(*dict(back, **kw).values())  # noqa: E731
    assert b() == tst.TST_ERR_NO_DEVICE
    for kw in (dict(weight=None), dict(d_out=None), dict(d_rows=None), dict(d_weight=None), dict(rows=None), dict(d_out_ld=1)):
        assert b(**kw) == tst.TST_ERR_INVALID_ARG, kw
    assert b(d_rows=A16 + 1) == tst.TST_ERR_ALIGNMENT


def test_grouped_block_scaled_plan_rules():
    kw = dict(dtype="e4m3", host_only=True, num_sms=152)
    p = tst.gemm_grouped_plan_create(8, 1000, 512, 1024, ab_block=(1, 128, 128), **kw)
    assert (p.info.bm, p.info.bn, p.info.cta_group, p.info.bk, p.info.tma_store) == (128, 128, 1, 128, 0)
    # the form by the sizes: few rows per group, many, or k-blocks that only the general form has
    for G, M, N, ab, bn, form in ((32, 64, 4096, (1, 128, 128), 0, (16, 128)), (32, 1024, 4096, (1, 128, 128), 0, (32, 128)),
                                  (32, 1024, 4096, (1, 128, 1), 0, (32, 128)), (16, 16384, 4096, (1, 128, 128), 0, (128, 256)),
                                  (16, 16384, 4096, (1, 128, 64), 0, (128, 128)), (16, 16384, 100, (1, 128, 128), 0, (128, 128)),
                                  (32, 64, 4096, (1, 64, 128), 0, (128, 128)), (600, 600, 4096, (1, 128, 128), 0, (128, 128)),
                                  (32, 64, 4096, (1, 128, 128), 128, (128, 128)), (4, 64, 4096, (1, 128, 128), 256, (128, 256))):
        info = tst.gemm_grouped_plan_create(G, M, N, 1024, ab_block=ab, bn=bn, **kw).info
        assert (info.bm, info.bn) == form, (G, M, N, ab, bn)
    assert tst.gemm_plan_create(1000, 1000, 1024, schedule="persistent", ab_block=(1, 128, 128), bn=256, **kw).info.bn == 256
    for bad, status in ((dict(dtype="bf16"), tst.TST_ERR_UNSUPPORTED), (dict(bn=512), tst.TST_ERR_UNSUPPORTED),
                        (dict(bn=256, ab_block=(1, 128, 64)), tst.TST_ERR_UNSUPPORTED), (dict(stages=7), tst.TST_ERR_UNSUPPORTED),
                        (dict(cta_group=2), tst.TST_ERR_UNSUPPORTED), (dict(activation="gelu"), tst.TST_ERR_UNSUPPORTED),
                        (dict(out_dtype="e4m3"), tst.TST_ERR_UNSUPPORTED), (dict(ab_block=(1, 100)), tst.TST_ERR_INVALID_ARG)):
        with pytest.raises(tst.TstError) as e:
            tst.gemm_grouped_plan_create(8, 1000, 512, 1024, **dict(dict(kw, ab_block=(1, 128, 128)), **bad))
        assert e.value.status == status, bad
