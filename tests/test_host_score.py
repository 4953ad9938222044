"""Routing by scores and int8 rows without a GPU: plan rules and refusals at the C boundary (host-only plans;
no kernel runs)."""
import ctypes

import pytest

import tile_scheduled_tensor_gb300 as tst


def _plan(T=100, E=64, k=8, **kw):
    return tst.moe_plan_create(T, E, k, host_only=True, **dict(dict(score="sigmoid", groups=8, top_groups=4, group_best=2), **kw))


def test_plan_rules():
    invalid, unsupported = tst.TST_ERR_INVALID_ARG, tst.TST_ERR_UNSUPPORTED
    info = tst.moe_plan_get_info(_plan(normalize=False, balance_coef=0.5))
    assert (info.max_tokens, info.experts, info.top_k, info.normalize, info.balance_coef) == (100, 64, 8, 0, 0.5)
    for kw, status in ((dict(T=0), invalid), (dict(E=60), invalid), (dict(groups=0), invalid), (dict(top_groups=0), invalid), (dict(top_groups=9), invalid),
                       (dict(group_best=0), invalid), (dict(group_best=3), invalid), (dict(k=33), unsupported), (dict(top_groups=1, k=9), invalid),
                       (dict(groups=64, top_groups=32, group_best=2), invalid), (dict(score=2), invalid), (dict(weight_scale=float("nan")), invalid),
                       (dict(weight_scale=float("inf")), invalid), (dict(balance_coef=float("nan")), invalid),
                       (dict(groups=64, top_groups=32, group_best=1), unsupported), (dict(E=1028, groups=4), unsupported),
                       (dict(E=1023, groups=3, top_groups=2), unsupported), (dict(k=33, groups=1, top_groups=1), unsupported)):
        with pytest.raises(tst.TstError) as e:
            _plan(**kw)
        assert e.value.status == status, kw
    _plan(E=1024, groups=32, top_groups=1), _plan(E=768, groups=3, top_groups=1), _plan(E=1, k=1, groups=1, top_groups=None, group_best=1)
    for kw in (dict(groups=2), dict(top_groups=2), dict(group_best=2), dict(weight_scale=2.0)):
        with pytest.raises(ValueError):
            tst.moe_plan_create(4, 8, 2, host_only=True, **kw)
    with pytest.raises(ValueError):
        _plan(score="tanh")
    assert tst.lib.moe_plan_create_scored(None, 4, 8, 2, None) == invalid
    h = ctypes.c_void_p(1)
    assert tst.lib.moe_plan_create_scored(ctypes.byref(h), 4, 8, 2, None) == invalid and not h.value


# addresses that are only checked, never read: a host-only plan stops before any launch
A16, A8, A4, A2 = 1 << 20, (1 << 20) + 8, (1 << 20) + 4, (1 << 20) + 2
F32, BF16, INT8 = tst.TST_OUT_F32, tst.TST_OUT_BF16, tst.TST_OUT_INT8


def test_route_refusals():
    p, plain = _plan(), tst.moe_plan_create(100, 64, 8, host_only=True)
    good = dict(plan=p._h, tokens=10, logits=A16, dtype=F32, ld=64, mask=None, bias=None, expert=A4, weight=A4, row=A4, counts=A4,
                totals=A4, loss=A4, stream=None)
    call = lambda **kw: tst.lib.moe_route_scored(*dict(good, **kw).values())  # noqa: E731
    assert call() == tst.TST_ERR_NO_DEVICE and call(bias=A4, tokens=0, logits=None, expert=None) == tst.TST_ERR_NO_DEVICE
    for kw in (dict(plan=None), dict(plan=plain._h), dict(tokens=-1), dict(tokens=101), dict(dtype=INT8), dict(dtype=7), dict(ld=63),
               dict(logits=None), dict(expert=None), dict(weight=None), dict(row=None), dict(counts=None), dict(totals=None), dict(loss=None)):
        assert call(**kw) == tst.TST_ERR_INVALID_ARG, kw
    for kw in (dict(logits=A2), dict(dtype=BF16, logits=A2 + 1), dict(expert=A2), dict(loss=A2), dict(bias=A2)):
        assert call(**kw) == tst.TST_ERR_ALIGNMENT, kw
    # a plan with a score has no plain routing
    assert tst.lib.moe_route(p._h, 10, A16, F32, 64, None, A4, A4, A4, A4, A4, A4, None) == tst.TST_ERR_INVALID_ARG
    grad = dict(plan=p._h, tokens=10, logits=A16, dtype=F32, ld=64, mask=None, expert=A4, counts=A4, totals=A4, d_weight=None,
                d_loss=None, d_logits=A16, d_ld=64, stream=None)
    back = lambda **kw: tst.lib.moe_route_scored_backward(*dict(grad, **kw).values())  # noqa: E731
    assert back() == tst.TST_ERR_NO_DEVICE
    assert tst.lib.moe_route_backward(*grad.values()) == tst.TST_ERR_INVALID_ARG
    for kw in (dict(plan=plain._h), dict(d_ld=63), dict(d_logits=None), dict(expert=None), dict(counts=None), dict(totals=None), dict(tokens=101)):
        assert back(**kw) == tst.TST_ERR_INVALID_ARG, kw
    assert back(d_logits=A2) == tst.TST_ERR_ALIGNMENT and back(d_loss=A2) == tst.TST_ERR_ALIGNMENT


def test_int8_row_refusals():
    p = _plan()
    disp = dict(plan=p._h, tokens=10, hidden=64, x=A16, x_dtype=BF16, x_ld=64, row=A4, rows=A16, rows_dtype=INT8, n_rows=80,
                scales=A4, stream=None)
    d = lambda **kw: tst.lib.moe_dispatch(*dict(disp, **kw).values())  # noqa: E731
    assert d() == tst.TST_ERR_NO_DEVICE and d(row=None) == tst.TST_ERR_NO_DEVICE and d(x=A2) == tst.TST_ERR_NO_DEVICE
    for kw in (dict(hidden=0), dict(x_ld=63), dict(x_dtype=INT8), dict(rows_dtype=4), dict(x=None), dict(rows=None), dict(scales=None), dict(n_rows=-1),
               dict(tokens=101), dict(row=None, n_rows=9), dict(row=None, tokens=801)):
        assert d(**kw) == tst.TST_ERR_INVALID_ARG, kw
    for kw in (dict(hidden=72, x_ld=72), dict(rows=A8), dict(x=A16 + 1), dict(scales=A2)):
        assert d(**kw) == tst.TST_ERR_ALIGNMENT, kw
