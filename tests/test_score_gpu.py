"""GPU parity of routing by scores (moe_route and moe_route_backward on a plan with a score) and of the int8
rows of moe_dispatch against the FP64 oracle.

Whole numbers (experts, rows, counts, int8 values) are equal.  With u = 2^-24:
  sigmoid       1 / (1 + e^-l): e^-l from ex2 of a rounded product, (1.5 |l| + 3) u relative for |l| < 80, and 8 u of
                the sum and the quotient
  weights       a quotient of two such, times the scale; e^x of the chosen logits: (2.4 |l - top| + 1.5 |l| + 40) u
  loss          shares of such scores, summed as moe_route's: (200 + 3 |l| + 4 log2 E + T / 8192 + E / 256) u
  d_logits      terms that carry such errors twice: (512 + 4 |l|) u of the sum of magnitudes, and half a unit in the
                last place of a BF16 result; what underflows FP32 is below 2^-120"""
import numpy as np
import pytest
import torch

import tile_scheduled_tensor_gb300 as tst
from oracle import moe

from gemm_check import half_ulp_bf16

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def _dev(x, dtype="f32"):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).cuda().to(TYPES[dtype])


def _host(x):
    return x.float().cpu().numpy().astype(np.float64)


def _strided(x, pad):
    """The same values as rows of a wider tensor whose other columns are NaN."""
    wide = torch.full((x.shape[0], x.shape[1] + pad), float("nan"), dtype=x.dtype, device=x.device)
    wide[:, :x.shape[1]] = x
    return wide[:, :x.shape[1]]


def _route(plan, logits, bias=None, mask=None, stream=None):
    T, k, E = logits.shape[0], plan.top_k, plan.experts
    i32 = dict(dtype=torch.int32, device="cuda")
    o = dict(expert=torch.full((T, k), -7, **i32), weight=torch.full((T, k), float("nan"), device="cuda"),
             row=torch.full((T, k), -7, **i32), counts=torch.full((E,), -7, **i32), totals=torch.full((2,), -7, **i32),
             loss=torch.full((1,), float("nan"), device="cuda"))
    if stream is not None:
        torch.cuda.synchronize()
    tst.moe_route(plan, logits, o["expert"], o["weight"], o["row"], o["counts"], o["totals"], o["loss"], mask=mask, bias=bias, stream=stream)
    return o


def _check(o, want, l):
    for name in ("expert", "row", "counts", "totals"):
        assert np.array_equal(o[name].cpu().numpy(), want[name]), name
    T, E = l.shape
    e = want["expert"]
    at = np.take_along_axis(l, np.maximum(e, 0), 1)
    at = np.where((e >= 0) & np.isfinite(at), at, 0.0)
    spread = np.minimum(np.abs(at.max(axis=1, keepdims=True) - at.min(axis=1, keepdims=True)), 104.0)
    top = np.minimum(np.abs(np.where(np.isfinite(l), l, 0.0)).max(axis=1, keepdims=True), 88.0)   # beyond, e^l is 0 or 1
    got = _host(o["weight"])
    assert np.array_equal(np.isnan(got), np.isnan(want["weight"]))
    ok = ~np.isnan(got)
    tol = (2.4 * (spread + top) + 1.5 * np.minimum(np.abs(at), 88.0) + 40) * U * np.abs(want["weight"]) + 2.0 ** -120
    assert (np.abs(got - want["weight"]) <= tol)[ok].all(), float(np.max((np.abs(got - want["weight"]) - tol)[ok]))
    loss, ref = o["loss"].item(), want["loss"]
    if np.isnan(ref):
        assert np.isnan(loss)
    else:
        assert abs(loss - ref) <= (200 + 3 * top.max() + 4 * np.log2(E) + T / 8192 + E / 256) * U * abs(ref) + 1e-30, (loss, ref)


def _case(seed, T, E, bias=True, spread=1.0):
    rng = np.random.default_rng(seed)
    l = rng.normal(size=(T, E)) * spread + 0.5 * rng.normal(size=E)[None, :]
    return l, (0.001 * rng.integers(-100, 101, E)).astype(np.float32) if bias else None


# experts, groups and choices on each side of the kernels' widths: one expert, groups of one, odd groups, three and five
# groups (lanes without a group), every expert chosen, few lanes left by the groups, whole and ragged packs
SHAPES = [(1, 1, 1, 1, 1, 1), (1, 256, 8, 8, 4, 2), (2, 2, 2, 2, 2, 1), (7, 6, 3, 3, 2, 2), (33, 8, 2, 4, 1, 2), (64, 31, 31, 1, 1, 1),
          (65, 32, 4, 32, 8, 1), (100, 33, 6, 11, 5, 2), (257, 60, 4, 4, 3, 1), (300, 64, 8, 8, 4, 2), (511, 100, 10, 5, 2, 2),
          (256, 129, 7, 3, 2, 2), (400, 256, 8, 8, 4, 2), (130, 257, 32, 1, 1, 1), (60, 512, 8, 8, 1, 2), (40, 510, 16, 30, 7, 2),
          (50, 640, 10, 5, 5, 1), (70, 1024, 16, 16, 4, 2), (35, 1024, 32, 32, 1, 1), (90, 160, 6, 8, 3, 1), (128, 384, 5, 1, 1, 1)]


@pytest.mark.parametrize("T,E,k,G,g,best", SHAPES)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_route_equals_the_oracle(T, E, k, G, g, best, dtype, score):
    for normalize, use_bias in ((True, True), (False, False)):
        l, bias = _case(T + E + G, T, E, use_bias)
        logits = _dev(l, dtype)
        l = _host(logits)
        plan = tst.moe_plan_create(T + 3, E, k, normalize=normalize, balance_coef=0.02, score=score, groups=G, top_groups=g, group_best=best,
                                   weight_scale=2.5)
        want = moe.route_scored(l, k, score == "sigmoid", bias, G, g, best, normalize, 2.5, 0.02)
        _check(_route(plan, logits, None if bias is None else _dev(bias)), want, l)


def _settled(l, bias, G, g):
    """Rows whose kept groups, by sums of two softmax scores, do not hang on a rounding.  (x + b) + (y + d) and (x + d) + (y + b) are one number
    and two roundings of it: scores are within 2 u' of the formula's (u' = 2^-53, values up to 2), the sums add
    2 u' each, so values within 2^-48 = 32 u' of the last one kept have to come of the same logits and biases."""
    size, out = l.shape[1] // G, np.ones(len(l), dtype=np.uint8)
    for t in range(len(l)):
        c = np.where(l[t] > -np.inf, moe.scores(l[t], False) + bias, -np.inf)
        best = [sorted(range(i * size, (i + 1) * size), key=lambda e: (-c[e], e))[:2] for i in range(G)]
        groups = sorted(((sum(c[e] for e in b if c[e] > -np.inf), sorted((l[t, e], bias[e]) for e in b if c[e] > -np.inf))
                         for b in best if c[b[0]] > -np.inf), key=lambda v: -v[0])
        if len(groups) > g:
            value, of = groups[g - 1]
            out[t] = all(o == of for v, o in groups if abs(v - value) < 2.0 ** -48)
    return out


@pytest.mark.parametrize("E,k,G,g,best", [(256, 8, 8, 4, 2), (64, 6, 8, 3, 1), (60, 4, 5, 2, 2), (48, 5, 16, 7, 2), (96, 32, 1, 1, 1), (20, 3, 1, 1, 1)])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("kind", ["zeros", "levels", "closed", "saturated"])
def test_rows_whose_values_tie_or_nearly(E, k, G, g, best, score, kind):
    """Choices among equal values and among neighbours in FP32: every row is chosen by FP64 values, or by rounds where
    more than the list holds are in reach.  Two levels a row, so that different sums of two are steps apart."""
    rng = np.random.default_rng(E + G + len(kind))
    T = 150
    l = np.zeros((T, E))
    if kind in ("levels", "closed"):
        base = np.float32(rng.normal(size=(T, 1)))
        l = np.where(rng.random((T, E)) < 0.5, base, np.nextafter(base, np.float32(9))).astype(np.float64)
    if kind == "closed":   # groups with one open expert, or none
        l[rng.random((T, E)) < rng.choice([0.5, 0.9, 0.97], (T, 1))] = -np.inf
    if kind == "saturated":   # 1 / (1 + e^-l) is 1 in FP64 from 37 on
        l = rng.choice([36.0, 38.0, 50.0], (T, E))
    biases = [None, np.zeros(E), np.full(E, -0.75), rng.choice([-0.25, 0.0, 0.25], E)]
    if best == 2 and kind in ("levels", "closed"):   # (x + b) + (y + d) and (x + d) + (y + b) are apart by their roundings alone
        biases.pop()
    for bias in biases:
        bias = None if bias is None else bias.astype(np.float32)
        logits = _dev(l)
        plan = tst.moe_plan_create(T, E, k, normalize=False, score=score, groups=G, top_groups=g, group_best=best, balance_coef=0.5)
        mask = np.ones(T, dtype=np.uint8)
        if best == 2 and score == "softmax":   # (the sigmoids here have one rounding: 1/2, 1 and 1 - 2^-52, or two levels)
            mask = _settled(l, np.zeros(E) if bias is None else bias.astype(np.float64), G, g)
        assert mask.sum() >= T // 2
        want = moe.route_scored(_host(logits), k, score == "sigmoid", bias, G, g, best, False, 1.0, 0.5, mask=mask)
        _check(_route(plan, logits, None if bias is None else _dev(bias), mask=torch.from_numpy(mask).cuda()), want, _host(logits))


@pytest.mark.parametrize("T", [31, 32, 33, 2000, 4865, 9728, 19457])
def test_many_chunks(T):
    E, k = 24, 3
    l, bias = _case(T, T, E)
    logits = _dev(l + np.linspace(0, 2, E)[None, :])
    l = _host(logits)
    plan = tst.moe_plan_create(50000, E, k, balance_coef=1.0, score="sigmoid", groups=4, top_groups=2, group_best=2)
    want = moe.route_scored(l, k, True, bias, 4, 2, 2, True, 1.0, 1.0)
    for _ in range(2):   # the plan's workspace again
        _check(_route(plan, logits, _dev(bias)), want, l)


@pytest.mark.parametrize("T,E,k,G,dtype,score,kind", [
    (9800, 256, 8, 8, "f32", "sigmoid", "normal"), (9800, 256, 8, 8, "bf16", "sigmoid", "ties"), (9733, 60, 4, 4, "bf16", "softmax", "masked"),
    (9729, 128, 8, 1, "f32", "softmax", "ties"), (9728, 64, 6, 8, "f32", "sigmoid", "masked"), (9728, 96, 4, 3, "f32", "softmax", "equal"),
    (9728, 64, 8, 8, "bf16", "sigmoid", "equal"), (9728, 128, 8, 4, "f32", "sigmoid", "close"), (9728, 128, 8, 4, "f32", "softmax", "close")])
def test_many_tokens(T, E, k, G, dtype, score, kind):
    rng = np.random.default_rng(T + E)
    l, bias = _case(5 + E, T, E)
    mask = None
    if kind == "ties":
        l, bias = np.round(l * 2) / 2, np.round(bias * 20).astype(np.float32) / 20
    elif kind == "equal":
        l[:], bias = 0.25, None
    elif kind == "close":   # values that FP32 scores cannot tell apart: neighbouring logits, and biases that make up for them
        l = 1.0 + rng.integers(0, 64, (T, E)) * 2.0 ** -23
        bias = (rng.integers(-4, 5, E) * 2.0 ** -24).astype(np.float32)
    elif kind == "masked":
        l[rng.random((T, E)) < 0.3] = -np.inf
        l[rng.random(T) < 0.05] = -np.inf        # nothing open
        l[7:40, 2:] = -np.inf                    # fewer open than k
        mask = (rng.random(T) < 0.9).astype(np.uint8)
    logits = _dev(l, dtype)
    l = _host(logits)
    plan = tst.moe_plan_create(T, E, k, normalize=kind != "masked", balance_coef=0.5, score=score, groups=G, top_groups=max(1, G // 2), group_best=2)
    want = moe.route_scored(l, k, score == "sigmoid", bias, G, max(1, G // 2), 2, kind != "masked", 1.0, 0.5, mask)
    m = None if mask is None else torch.from_numpy(mask).cuda()
    if m is not None:
        logits[m == 0] = float("nan")
        logits = _strided(logits, 8)
        l = np.where(np.asarray(mask)[:, None] != 0, l, 0.0)
    _check(_route(plan, logits, None if bias is None else _dev(bias), m), want, l)


@pytest.mark.parametrize("shift", [-1e4, -300.0, -95.0, -50.0, 30.0, 80.0, 1e4, 3e38])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("use_bias", [True, False])
def test_every_finite_logit_gives_finite_results(shift, score, use_bias):
    T, E, k = 70, 48, 4
    l, bias = _case(11, T, E, use_bias)
    logits = _dev(l + shift if abs(shift) < 1e38 else np.where(l > 0, shift, -shift))
    l = _host(logits)
    want = moe.route_scored(l, k, score == "sigmoid", bias, 4, 2, 1, True, 1.0, 0.5)
    plan = tst.moe_plan_create(T, E, k, normalize=True, balance_coef=0.5, score=score, groups=4, top_groups=2)
    o = _route(plan, logits, None if bias is None else _dev(bias))
    assert torch.isfinite(o["weight"]).all() and torch.isfinite(o["loss"]).all()
    _check(o, want, l)
    dw = np.random.default_rng(1).normal(size=(T, k))
    d = torch.empty_like(logits)
    tst.moe_route_backward(plan, logits, o["expert"], o["counts"], o["totals"], d, d_weight=_dev(dw), d_loss=torch.ones(1, device="cuda"))
    ref, size = moe.route_scored_backward(l, _host(_dev(dw)), 1.0, want, score == "sigmoid", True, 1.0, 0.5)
    # a product with 1 - s of a large logit is 0 in FP32 below 2^-126; e^l of a logit past 80 in magnitude weighs nothing beside its neighbours'
    assert (np.abs(_host(d) - ref) <= (512 + 4 * 88) * U * size + 2.0 ** -100).all()


def test_infinite_and_missing_values():
    # +inf and NaN logits and biases count as +inf; a bias of -inf is never chosen; a closed expert neither
    T, E, k = 6, 8, 3
    l = np.tile(np.linspace(-1, 1, E), (T, 1))
    l[1, 2], l[2, 5], l[3, 6], l[4] = np.nan, np.inf, -np.inf, -np.inf
    l[4, 1] = 0.0
    for score in ("sigmoid", "softmax"):
        for bias in (None, np.array([0, 0, 0, -np.inf, 0, 0, 0, -np.inf], np.float32), np.array([np.inf, 0, np.nan, 0, 0, 0, 0, 0], np.float32)):
            want = moe.route_scored(l, k, score == "sigmoid", bias, 2, 1, 1, True, 1.0, 0.5)
            plan = tst.moe_plan_create(T, E, k, balance_coef=0.5, score=score, groups=2, top_groups=1)
            o = _route(plan, _dev(l), None if bias is None else _dev(bias))
            for name in ("expert", "row", "counts", "totals"):
                assert np.array_equal(o[name].cpu().numpy(), want[name]), (score, bias, name)
            rows = [0, 3, 4, 5]
            assert np.allclose(_host(o["weight"])[rows], want["weight"][rows], rtol=1e-5, atol=0)


def test_no_tokens_and_nothing_open():
    plan = tst.moe_plan_create(64, 16, 2, balance_coef=0.5, score="sigmoid", groups=4, top_groups=2)
    for T in (0, 5, 40):
        o = _route(plan, torch.full((T, 16), float("-inf"), device="cuda"), torch.zeros(16, device="cuda"))
        assert (o["expert"] == -1).all() and (o["row"] == -1).all() and not o["weight"].any()
        assert not o["counts"].any() and o["totals"].tolist() == [0, 0] and o["loss"].item() == 0.0


GRADS = [(1, 256, 8, 8, "f32"), (33, 60, 4, 4, "bf16"), (200, 129, 7, 3, "f32"), (130, 257, 32, 1, "bf16"), (65, 31, 5, 1, "f32"),
         (70, 1024, 16, 16, "f32"), (3000, 96, 6, 8, "f32"), (90, 510, 16, 30, "bf16"), (50, 2, 2, 1, "f32"), (40, 1, 1, 1, "f32")]


@pytest.mark.parametrize("T,E,k,G,dtype", GRADS)
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("normalize", [True, False])
def test_gradient_equals_the_oracle(T, E, k, G, dtype, score, normalize):
    rng = np.random.default_rng(T + E)
    l, bias = _case(T, T, E)
    mask = None
    if T > 30:
        l[rng.random((T, E)) < 0.1] = -np.inf
        mask = (rng.random(T) < 0.9).astype(np.uint8)
    logits = _dev(l, dtype)
    l = _host(logits)
    g, sig = max(1, G // 2), score == "sigmoid"
    if k > g * (E // G):
        g = G
    plan = tst.moe_plan_create(T, E, k, normalize=normalize, balance_coef=0.5, score=score, groups=G, top_groups=g, weight_scale=2.5)
    want = moe.route_scored(l, k, sig, bias, G, g, 1, normalize, 2.5, 0.5, mask)
    m = None if mask is None else torch.from_numpy(mask).cuda()
    if T % 2:
        logits = _strided(logits, 5)
    o = _route(plan, logits, _dev(bias), m)
    assert np.array_equal(o["expert"].cpu().numpy(), want["expert"])
    dw, dl = _dev(rng.normal(size=(T, k))), _dev(np.array([0.7]))
    for use_w, use_l in ((True, True), (True, False), (False, True), (False, False)):
        d = _strided(torch.full((T, E), float("nan"), dtype=TYPES[dtype], device="cuda"), 3)
        tst.moe_route_backward(plan, logits, o["expert"], o["counts"], o["totals"], d, d_weight=dw if use_w else None,
                               d_loss=dl if use_l else None, mask=m)
        ref, size = moe.route_scored_backward(l, _host(dw) * use_w, float(_host(dl)[0]) * use_l, want, sig, normalize, 2.5, 0.5, mask)
        tol = (512 + 4 * 8) * U * size + 2.0 ** -120
        if dtype == "bf16":
            tol = tol + half_ulp_bf16(ref) * 1.01
        assert (np.abs(_host(d) - ref) <= tol).all(), float((np.abs(_host(d) - ref) - tol).max())


def test_gradient_by_differences():
    # the FP32 weights and loss of the routing call itself, differenced with steps of 2^-7 (choices kept: far apart)
    T, E, k = 4, 12, 3
    l = np.linspace(-1.5, 1.5, E)[None, :] * np.array([1.0, -1.0, 0.7, -0.4])[:, None]
    for score in ("sigmoid", "softmax"):
        plan = tst.moe_plan_create(T, E, k, normalize=True, balance_coef=2.0, score=score, groups=3, top_groups=2, weight_scale=1.5)
        dw = np.random.default_rng(2).normal(size=(T, k))
        base = _route(plan, _dev(l))
        f = lambda x: (lambda o: float((_host(o["weight"]) * dw).sum() + o["loss"].item()))(_route(plan, _dev(x)))  # noqa: E731
        d = torch.empty(T, E, device="cuda")
        tst.moe_route_backward(plan, _dev(l), base["expert"], base["counts"], base["totals"], d, d_weight=_dev(dw), d_loss=torch.ones(1, device="cuda"))
        d, h = _host(d), 2.0 ** -7
        for t in range(T):
            for e in range(E):
                up, down = l.copy(), l.copy()
                up[t, e] += h
                down[t, e] -= h
                # third derivatives of at most 2 |dw| 1.5: h^2 / 6 * 9 = 1e-4; rounding 100 u * 10 / h = 8e-3 at most
                assert abs((f(up) - f(down)) / (2 * h) - d[t, e]) < 8.1e-3


def test_streams_graphs_and_plans_apart():
    T, E, k = 500, 64, 6
    l, bias = _case(21, T, E)
    l2, _ = _case(22, T, E)
    plan = tst.moe_plan_create(T, E, k, balance_coef=0.5, score="sigmoid", groups=8, top_groups=3, group_best=2)
    other = tst.moe_plan_create(T, E, k, balance_coef=0.5, score="softmax", groups=4, top_groups=2)
    logits, b = _dev(l), _dev(bias)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(10):
        o1, o2 = _route(plan, logits, b, stream=s1), _route(other, logits, b, stream=s2)
    torch.cuda.synchronize()
    _check(o1, moe.route_scored(_host(logits), k, True, bias, 8, 3, 2, True, 1.0, 0.5), _host(logits))
    _check(o2, moe.route_scored(_host(logits), k, False, bias, 4, 2, 1, True, 1.0, 0.5), _host(logits))
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        tst.moe_route(plan, logits, o1["expert"], o1["weight"], o1["row"], o1["counts"], o1["totals"], o1["loss"], bias=b)
        d = torch.empty_like(logits)
        tst.moe_route_backward(plan, logits, o1["expert"], o1["counts"], o1["totals"], d, d_weight=o1["weight"], d_loss=o1["loss"])
    logits.copy_(_dev(l2))
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    want = moe.route_scored(_host(logits), k, True, bias, 8, 3, 2, True, 1.0, 0.5)
    _check(o1, want, _host(logits))
    ref, size = moe.route_scored_backward(_host(logits), _host(o1["weight"]), o1["loss"].item(), want, True, True, 1.0, 0.5)
    assert (np.abs(_host(d) - ref) <= 600 * U * size + 2.0 ** -120).all()


# ------------------------------------------------------------------ int8 rows
def _rows_of(T, k, seed, drop=0.0):
    rng = np.random.default_rng(seed)
    row = rng.permutation(T * k).astype(np.int32).reshape(T, k)
    row[rng.random((T, k)) < drop] = -1
    return row


@pytest.mark.parametrize("T,H,k", [(1, 16, 1), (1, 4096, 8), (5, 48, 2), (33, 512, 3), (40, 528, 2), (9, 1040, 4), (7, 2048, 2), (6, 2064, 2), (5, 4112, 1),
                                   (3, 8192, 2), (3, 8208, 2), (2, 20000, 3), (700, 272, 4)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_int8_rows_equal_the_oracle(T, H, k, dtype):
    rng = np.random.default_rng(T + H)
    x = _dev(rng.normal(size=(T, H)) * np.exp(rng.normal(size=(T, 1)) * 3), dtype)
    x[T // 2, :H // 2] = 0.0
    if T > 4:
        x[1] = 0.0                  # the least scale
        x[2] = 1e-38 if dtype == "f32" else 0.0
        x[3, 0] = 3e38              # the largest magnitudes
    row = _rows_of(T, k, T, 0.2)
    plan = tst.moe_plan_create(T + 2, 16, k)
    n = T * k + 3
    for src in (x, _strided(x, 8), _strided(x, 3)):   # whole 16-byte units, and not
        for r in (row, None):
            out = torch.full((n, H), 99, dtype=torch.int8, device="cuda")
            scales = torch.full((n,), -7.0, device="cuda")
            tst.moe_dispatch(plan, src, None if r is None else torch.from_numpy(r).cuda(), out, scales=scales)
            q, s = moe.quantize_int8(_host(x).astype(np.float32))
            want, ws = np.full((n, H), 99.0), np.full(n, -7.0, np.float32)
            at = np.arange(T)[:, None] if r is None else r
            for j in range(at.shape[1]):
                has = at[:, j] >= 0
                want[at[has, j]], ws[at[has, j]] = q[has], s[has]
            assert np.array_equal(out.cpu().numpy(), want.astype(np.int8)) and np.array_equal(scales.cpu().numpy(), ws)
    assert tst.moe_status_query(plan) == tst.TST_OK


def test_int8_rows_of_no_numbers_and_of_no_place():
    x = torch.ones(4, 64, device="cuda")
    x[1, 3], x[2, 5] = float("nan"), float("inf")
    plan = tst.moe_plan_create(4, 16, 1)
    row = torch.tensor([[0], [1], [2], [9]], dtype=torch.int32, device="cuda")   # 9: past the matrix
    out, scales = torch.zeros(4, 64, dtype=torch.int8, device="cuda"), torch.full((4,), 5.0, device="cuda")
    tst.moe_dispatch(plan, x, row, out, scales=scales)
    assert tst.moe_status_query(plan) == tst.TST_ERR_DEVICE_CHECK
    s = scales.tolist()
    assert s[0] == np.float32(1) / np.float32(127) and np.isnan(s[1]) and np.isinf(s[2]) and s[3] == 5.0 and not out[3].any()


# ------------------------------------------------------------------ the calls of a layer together
@pytest.mark.parametrize("T,E,k,H,inner", [(1, 16, 4, 256, 192), (50, 16, 4, 256, 192), (600, 8, 2, 512, 272), (3, 32, 3, 1040, 64)])
def test_a_layer_in_int8(T, E, k, H, inner):
    """route -> dispatch -> grouped product with ReLU -> dispatch -> grouped product -> combine, each step from the library's
    own results of the step before.  The int8 values equal the oracle's; the products lie within their bounds."""
    from oracle import int8
    rng = np.random.default_rng(T + E)
    l, bias = _case(T + 1, T, E)
    x = _dev(rng.normal(size=(T, H)), "bf16")
    up, us = moe.quantize_int8(rng.normal(size=(E * inner, H)).astype(np.float32))
    down, ds = moe.quantize_int8(rng.normal(size=(E * H, inner)).astype(np.float32))
    i8 = lambda v: torch.from_numpy(v.astype(np.int8)).cuda()  # noqa: E731
    plan = tst.moe_plan_create(T, E, k, score="sigmoid", groups=4, top_groups=2, group_best=2, weight_scale=2.5)
    o = _route(plan, _dev(l), _dev(bias))
    R = T * k
    a, sa = torch.zeros(R, H, dtype=torch.int8, device="cuda"), torch.zeros(R, device="cuda")
    mid, b, sb = torch.empty(R, inner, dtype=torch.bfloat16, device="cuda"), torch.zeros(R, inner, dtype=torch.int8, device="cuda"), torch.zeros(R, device="cuda")
    rows, out = torch.empty(R, H, dtype=torch.bfloat16, device="cuda"), torch.empty(T, H, device="cuda")
    p1 = tst.gemm_int8_plan_create(R, inner, H, groups=E, relu=True)
    p2 = tst.gemm_int8_plan_create(R, H, inner, groups=E)
    tst.moe_dispatch(plan, x, o["row"], a, scales=sa)
    tst.gemm_int8_run(p1, a, i8(up), mid, sa, _dev(us), group_rows=o["counts"])
    tst.moe_dispatch(plan, mid, None, b, scales=sb)
    tst.gemm_int8_run(p2, b, i8(down), rows, sb, _dev(ds), group_rows=o["counts"])
    tst.moe_combine(plan, rows, o["row"], out, weight=o["weight"])
    want = moe.route_scored(_host(_dev(l)), k, True, bias, 4, 2, 2, True, 2.5, 0.01)
    for name in ("expert", "row", "counts"):
        assert np.array_equal(o[name].cpu().numpy(), want[name]), name
    q, s = moe.quantize_int8(_host(x).astype(np.float32))
    token = np.empty(R, dtype=np.int64)
    token[want["row"].reshape(-1)] = np.repeat(np.arange(T), k)
    assert np.array_equal(a.cpu().numpy(), q[token].astype(np.int8)) and np.array_equal(sa.cpu().numpy(), s[token])

    def product(A, S, B, C, D, relu):
        ref, size = int8.gemm(A.cpu().numpy(), B, _host(S), C, None, relu, want["counts"].tolist())
        assert (np.abs(_host(D) - ref) <= 2.01 * U * size + 1.01 * U * np.abs(ref) + 1.01 * half_ulp_bf16(ref)).all()
    product(a, sa, up, us, mid, True)
    qm, sm = moe.quantize_int8(_host(mid).astype(np.float32))
    assert np.array_equal(b.cpu().numpy(), qm.astype(np.int8)) and np.array_equal(sb.cpu().numpy(), sm)
    product(b, sb, down, ds, rows, False)
    ref, size = moe.combine(_host(rows), want["row"], _host(o["weight"]))
    assert (np.abs(_host(out) - ref) <= (k + 1) * U * size).all()
    for p in (p1, p2):
        assert tst.gemm_int8_status_query(p) == tst.TST_OK
