"""GPU parity of the calls around a mixture of experts (moe_route, moe_route_backward,
moe_dispatch, moe_combine, moe_combine_backward) against the FP64 oracle.

Whole numbers (experts, rows, counts) and e4m3 values are equal; floating results lie within
bounds from the number formats, with u = 2^-24 the unit roundoff of FP32:
  weights       __expf is within 2 + 1.16 |x| units in the last place (2u) of e^x; a weight is a
                quotient of it and a sum of E of them (sum error below (log2 E + 6) u), and the sum's
                terms weigh |x| by e^x, at most log E + 1 on average: in all
                (4 + 2.4 |x| + 4 (log2 E + 2) + 12) u relative
  loss          a probability's error as above, and sums of at most 256 / 8 + 8 + T / 8192 + 5 + E / 256
                + 13 terms in sequence: (160 + 4 log2 E + T / 8192 + E / 256) u relative
  d_logits      each of its terms carries such an error, twice over (a product of two): 256 u of the
                sum of magnitudes, and half a unit in the last place of a BF16 result
  combine       k products and sums: (k + 1) u of the sum of magnitudes, and the result's rounding
  d_rows        one product, rounded once or (BF16) twice
  d_weight      a dot product of H terms: (H / 256 + 24) u of the sum of magnitudes"""
import numpy as np
import pytest
import torch

import synthetic
import tile_scheduled_tensor_gb300 as tst
from oracle import moe

from gemm_check import half_ulp_bf16, host_values

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def _normal(seed, *shape):
    n = int(np.prod(shape))
    return synthetic.draw("normal", seed, n).reshape(shape) if n else np.zeros(shape)


def _dev(x, dtype="f32"):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).cuda().to(TYPES[dtype])


def _host(x):
    return x.float().cpu().numpy().astype(np.float64)


def _strided(x, pad):
    """The same values as rows of a wider tensor whose other columns are NaN."""
    wide = torch.full((x.shape[0], x.shape[1] + pad), float("nan"), dtype=x.dtype, device=x.device)
    wide[:, :x.shape[1]] = x
    return wide[:, :x.shape[1]]


def _route(plan, logits, mask=None):
    T, k, E = logits.shape[0], plan.top_k, plan.experts
    i32 = dict(dtype=torch.int32, device="cuda")
    o = dict(expert=torch.full((T, k), -7, **i32), weight=torch.full((T, k), float("nan"), device="cuda"),
             row=torch.full((T, k), -7, **i32), counts=torch.full((E,), -7, **i32), totals=torch.full((2,), -7, **i32),
             loss=torch.full((1,), float("nan"), device="cuda"))
    tst.moe_route(plan, logits, o["expert"], o["weight"], o["row"], o["counts"], o["totals"], o["loss"], mask=mask)
    return o


def _check_route(o, want, l, normalize):
    for name in ("expert", "row", "counts", "totals"):
        assert np.array_equal(o[name].cpu().numpy(), want[name]), name
    T, E = l.shape
    x = np.zeros(want["expert"].shape)
    for t in range(T):
        s = want["expert"][t] >= 0
        if s.any() and np.isfinite(l[t].max()):
            x[t, s] = np.minimum(l[t].max() - l[t, want["expert"][t][s]], 104.0)
    tol = (4 + 2.4 * x + 4 * (np.log2(E) + 2) + 12) * U
    got = _host(o["weight"])
    assert np.array_equal(np.isnan(got), np.isnan(want["weight"]))
    ok = ~np.isnan(got)
    # below 2^-126 a weight may be flushed or rounded to a subnormal
    assert (np.abs(got - want["weight"])[ok] <= (tol * want["weight"] + 2.0 ** -126)[ok]).all()
    loss, ref = o["loss"].item(), want["loss"]
    if np.isnan(ref):
        assert np.isnan(loss)
    else:
        assert abs(loss - ref) <= (160 + 4 * np.log2(E) + T / 8192 + E / 256) * U * abs(ref) + 1e-30, (loss, ref)


# experts on each side of the kernels' widths, odd ones, one expert, every expert chosen
SHAPES = [(1, 1, 1), (1, 128, 8), (2, 2, 2), (7, 5, 3), (33, 8, 2), (64, 31, 31), (65, 32, 1), (100, 33, 6), (257, 60, 4),
          (300, 64, 8), (511, 100, 10), (256, 129, 7), (513, 256, 8), (130, 257, 32), (40, 513, 8), (70, 1024, 16)]


@pytest.mark.parametrize("T,E,k", SHAPES)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_route_equals_the_oracle(T, E, k, dtype):
    for normalize in (True, False):
        logits = _dev(_normal(100 + T + E, T, E), dtype)
        plan = tst.moe_plan_create(T + 3, E, k, normalize=normalize, balance_coef=0.02)
        o = _route(plan, logits)
        l = _host(logits)
        _check_route(o, moe.route(l, k, normalize, 0.02), l, normalize)


@pytest.mark.parametrize("T", [31, 32, 33, 2000, 9728, 9729, 19456, 19457, 20000])
def test_route_many_chunks(T):
    # token counts on both sides of the chunk sizes, uneven loads; a plan made for more tokens
    E, k = 12, 3
    logits = _dev(_normal(200 + T, T, E) + np.linspace(0, 2, E)[None, :])
    plan = tst.moe_plan_create(50000, E, k, balance_coef=1.0)
    l = _host(logits)
    want = moe.route(l, k, True, 1.0)
    for _ in range(2):
        _check_route(_route(plan, logits), want, l, True)


# many tokens per block: both types, whole and ragged rows, few and many choices
@pytest.mark.parametrize("T,E,k,dtype,kind", [
    (19456, 256, 8, "f32", "normal"), (19457, 200, 5, "bf16", "normal"), (20001, 64, 16, "f32", "normal"),
    (19999, 129, 8, "f32", "normal"), (19700, 255, 10, "bf16", "normal"), (19456, 40, 3, "bf16", "normal"),
    (19456, 512, 10, "bf16", "normal"), (19456, 33, 1, "f32", "normal"), (19456, 96, 8, "f32", "masked"),
    (19999, 130, 6, "bf16", "masked"), (19500, 128, 7, "f32", "ties"), (19500, 256, 8, "bf16", "ties"),
    (19456, 64, 8, "f32", "equal"), (70000, 34, 2, "f32", "normal")])
def test_route_of_many_tokens_equals_the_oracle(T, E, k, dtype, kind):
    rng = np.random.default_rng(T + E)
    l, mask = _normal(220 + T + E, T, E) * 2 + np.linspace(0, 1, E)[None, :], None
    if kind == "ties":
        l = np.round(l)
    elif kind == "equal":
        l[:] = 0.5
    elif kind == "masked":
        l[rng.random((T, E)) < 0.3] = -np.inf
        l[rng.random(T) < 0.05] = -np.inf                      # nothing open
        l[7:40, 2:] = -np.inf                                  # fewer open than k
        l[100:130] = 3e38                                      # beyond the plain exponentials
        mask = (rng.random(T) < 0.9).astype(np.uint8)
    plan = tst.moe_plan_create(T, E, k, normalize=kind != "masked", balance_coef=0.5)
    logits = _dev(l, dtype)
    ll = _host(logits)
    m = None if mask is None else torch.from_numpy(mask).cuda()
    if m is not None:
        logits[m == 0] = float("nan")
        logits = _strided(logits, 8)
    want = moe.route(ll, k, kind != "masked", 0.5, mask)
    if mask is not None:
        ll[mask == 0] = -np.inf
    first = _route(plan, logits, m)
    _check_route(first, want, ll, kind != "masked")
    again = _route(plan, logits, m)
    assert all(torch.equal(first[n], again[n]) for n in first)


def test_route_of_many_tokens_keeps_nan_and_infinities_visible():
    T, E, k = 19456, 64, 4
    l = _normal(230, T, E)
    l[11, 4] = np.nan
    l[12, 63] = np.inf
    l[13, 7] = l[13, 2] = np.nan
    l[19000] = np.nan
    plan = tst.moe_plan_create(T, E, k)
    o = _route(plan, _dev(l))
    want = moe.route(l.astype(np.float32).astype(np.float64), k, True, 0.01)
    _check_route(o, want, l.astype(np.float32).astype(np.float64), True)
    assert np.isnan(o["loss"].item()) and np.isnan(_host(o["weight"])[[11, 12, 13, 19000]]).all()


def test_route_masks_ties_and_closed_experts():
    T, E, k = 200, 24, 4
    rng = np.random.default_rng(3)
    l = rng.integers(-2, 3, (T, E)).astype(np.float64)        # many ties
    l[rng.random((T, E)) < 0.5] = -np.inf                      # closed experts, some rows with fewer than k open
    l[5] = -np.inf                                             # nothing open
    l[6] = np.finfo(np.float32).min                            # the type's lowest value everywhere: still open
    l[7] = -np.inf
    l[7, 3] = np.finfo(np.float32).min
    l[8] = 0.0
    l[8, ::2] = -0.0                                           # both zeros tie
    mask = (rng.random(T) < 0.8).astype(np.uint8)
    mask[5:9] = 1
    for dtype in ("f32", "bf16"):
        logits = _dev(l, dtype)
        if dtype == "bf16":
            logits[6] = torch.finfo(torch.bfloat16).min
            logits[7, 3] = torch.finfo(torch.bfloat16).min
        ll = _host(logits)
        logits[torch.from_numpy(mask).cuda() == 0] = float("nan")   # padding is never read
        for normalize in (True, False):
            plan = tst.moe_plan_create(T, E, k, normalize=normalize)
            for m in (torch.from_numpy(mask).cuda(), torch.from_numpy(mask).cuda().bool()):
                _check_route(_route(plan, logits, m), moe.route(ll, k, normalize, 0.01, mask), ll, normalize)


def test_route_everything_masked_and_no_tokens():
    plan = tst.moe_plan_create(64, 8, 2)
    o = _route(plan, torch.full((64, 8), float("nan"), device="cuda"), torch.zeros(64, dtype=torch.uint8, device="cuda"))
    assert (o["expert"] == -1).all() and (o["row"] == -1).all() and (o["weight"] == 0).all()
    assert (o["counts"] == 0).all() and (o["totals"] == 0).all() and o["loss"].item() == 0.0
    o = _route(plan, torch.empty(0, 8, device="cuda"))
    assert (o["counts"] == 0).all() and (o["totals"] == 0).all() and o["loss"].item() == 0.0


def test_route_nan_and_infinities_stay_visible():
    l = _normal(9, 6, 10)
    l[1, 4] = np.nan
    l[2, 3] = np.inf
    l[3, 7] = l[3, 2] = np.nan
    l[4, :] = np.nan
    logits = _dev(l)
    plan = tst.moe_plan_create(6, 10, 2)
    o = _route(plan, logits)
    want = moe.route(_host(logits), 2, True, 0.01)
    _check_route(o, want, _host(logits), True)
    assert np.isnan(o["loss"].item()) and np.isnan(_host(o["weight"])[1:5]).all()
    assert o["expert"][3].tolist() == [2, 7] and o["expert"][4].tolist() == [0, 1]


def test_route_strided_logits_other_stream_and_repeats():
    T, E, k = 700, 40, 5
    logits = _strided(_dev(_normal(10, T, E), "bf16"), 7)
    l = _host(logits)
    plan = tst.moe_plan_create(T, E, k)
    want = moe.route(l, k, True, 0.01)
    first = _route(plan, logits)
    _check_route(first, want, l, True)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        again = _route(plan, logits)
    torch.cuda.current_stream().wait_stream(s)
    for name in first:
        assert torch.equal(first[name], again[name]), name


@pytest.mark.parametrize("T,E,k", SHAPES)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_route_backward_equals_the_oracle(T, E, k, dtype):
    for normalize in (True, False):
        logits = _dev(_normal(300 + T + E, T, E), dtype)
        l = _host(logits)
        plan = tst.moe_plan_create(T, E, k, normalize=normalize, balance_coef=0.5)
        o = _route(plan, logits)
        r = moe.route(l, k, normalize, 0.5)
        dw = _dev(_normal(301 + T, T, k))
        d = torch.full_like(logits, float("nan"))
        tst.moe_route_backward(plan, logits, o["expert"], o["counts"], o["totals"], d, d_weight=dw,
                               d_loss=torch.tensor([0.75], device="cuda"))
        _check_grad(d, l, _host(dw), 0.75, r, normalize, 0.5, None, dtype)


def _check_grad(d, l, dw, d_loss, r, normalize, coef, mask, dtype):
    want, size = moe.route_backward(l, dw, d_loss, r, normalize, coef, mask)
    tol = 256 * U * size + 1e-37 + (half_ulp_bf16(want) if dtype == "bf16" else 0.0)
    err = np.abs(_host(d) - want)
    assert (err <= tol).all(), float(np.max(err / tol))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_route_backward_masks_and_missing_gradients(dtype):
    T, E, k = 150, 20, 4
    rng = np.random.default_rng(4)
    l = rng.standard_normal((T, E))
    l[rng.random((T, E)) < 0.6] = -np.inf
    l[3] = -np.inf
    mask = (rng.random(T) < 0.7).astype(np.uint8)
    logits = _dev(l, dtype)
    ll = _host(logits)
    m = torch.from_numpy(mask).cuda()
    logits[m == 0] = float("nan")
    logits = _strided(logits, 4)
    dw = rng.standard_normal((T, k)).astype(np.float32)
    for normalize in (True, False):
        plan = tst.moe_plan_create(T, E, k, normalize=normalize, balance_coef=0.1)
        o = _route(plan, logits, m)
        r = moe.route(ll, k, normalize, 0.1, mask)
        dead = (r["expert"] < 0)
        poisoned = _dev(dw)
        poisoned[torch.from_numpy(dead).cuda()] = float("nan")   # weights of no expert: their gradient is not read
        for w, g in ((poisoned, 0.3), (None, 0.3), (poisoned, None)):
            d = _strided(torch.full((T, E), float("nan"), dtype=TYPES[dtype], device="cuda"), 3)
            tst.moe_route_backward(plan, logits, o["expert"], o["counts"], o["totals"], d, d_weight=w, mask=m,
                                   d_loss=None if g is None else torch.tensor([g], device="cuda"))
            _check_grad(d, ll, np.zeros((T, k)) if w is None else np.where(dead, 0, dw).astype(np.float64), g or 0.0, r,
                        normalize, 0.1, mask, dtype)


def test_route_backward_against_differences_of_the_forward():
    # central differences of sum(dw * weight) + d_loss * loss, with the GPU's own forward in FP32:
    # step 2^-6, third-derivative error below step^2 / 6 * 4 of unit-sized terms, rounding 64 u / step
    T, E, k = 3, 6, 2
    base = _normal(12, T, E) * 2
    dw, plan = _normal(13, T, k), tst.moe_plan_create(T, E, k, balance_coef=0.5)
    logits = _dev(base)
    o = _route(plan, logits)
    d = torch.empty_like(logits)
    tst.moe_route_backward(plan, logits, o["expert"], o["counts"], o["totals"], d, d_weight=_dev(dw),
                           d_loss=torch.ones(1, device="cuda"))
    step = 2.0 ** -6

    def value(x):
        f = _route(plan, _dev(x))
        if not torch.equal(f["expert"], o["expert"]):
            return None
        return float((_host(f["weight"]) * dw).sum() + f["loss"].item())
    for t in range(T):
        for e in range(E):
            hi, lo = base.copy(), base.copy()
            hi[t, e] += step
            lo[t, e] -= step
            a, b = value(hi), value(lo)
            if a is None or b is None:   # the choice changed: no derivative there
                continue
            scale = np.abs(dw).sum() + 1
            assert abs((a - b) / (2 * step) - d[t, e].item()) <= scale * (step * step * 4 / 6 + 64 * U / step)


def test_calls_replay_from_a_cuda_graph():
    # captured once, replayed on new contents of the same tensors
    T, E, k, H = 300, 40, 3, 256
    plan = tst.moe_plan_create(T, E, k)
    logits, x = torch.empty(T, E, device="cuda"), torch.empty(T, H, device="cuda")
    o = _route(plan, logits.normal_())
    rows, out = torch.empty(T * k, H, device="cuda"), torch.empty(T, H, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        tst.moe_route(plan, logits, o["expert"], o["weight"], o["row"], o["counts"], o["totals"], o["loss"])
        tst.moe_dispatch(plan, x, o["row"], rows)
        tst.moe_combine(plan, rows, o["row"], out, weight=o["weight"])
    for seed in (1, 2):
        logits.copy_(_dev(_normal(240 + seed, T, E)))
        x.copy_(_dev(_normal(250 + seed, T, H)))
        graph.replay()
        _check_route(o, moe.route(_host(logits), k, True, 0.01), _host(logits), True)
        # the weights of a token add up to 1, so the copies come back as the token: k + 1 roundings
        # of parts of it, and k of the weights' own
        assert ((out - x).abs() <= (4 * k + 8) * 64 * U * x.abs()).all()


def _assign(T, k, E, seed, masked=False):
    """row (T x k) as routing gives it, and the number of rows."""
    rng = np.random.default_rng(seed)
    l = rng.standard_normal((T, E))
    mask = (rng.random(T) < 0.7).astype(np.uint8) if masked else None
    r = moe.route(l, k, True, 0.0, mask)
    return r["row"], int(r["totals"][0]), r["weight"].astype(np.float32)


@pytest.mark.parametrize("T,k,H", [(1, 1, 16), (1, 8, 4096), (5, 3, 128), (37, 2, 144), (64, 8, 512), (33, 4, 1040), (9, 6, 2064)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_dispatch_e4m3_equals_the_oracle(T, k, H, dtype):
    row, n, _ = _assign(T, k, 16, T + H, masked=T > 8)
    x = _dev(_normal(400 + T, T, H) * np.exp2(np.linspace(-20, 20, T))[:, None], dtype)
    x[0, :min(H, 128)] = 0                                     # a tile of zeros
    plan = tst.moe_plan_create(T, 16, k)
    want, scale = moe.quantize(_host(x).astype(np.float32))
    for src in (x, _strided(x, 16), _strided(x, 3)):           # vectors, and one element at a time
        q = torch.zeros(n, H, dtype=torch.uint8, device="cuda")
        s = torch.full((n, -(-H // 128)), float("nan"), device="cuda")
        tst.moe_dispatch(plan, src, torch.from_numpy(row).cuda(), q, scales=s)
        qv, sv = _host(q.view(torch.float8_e4m3fn)), s.cpu().numpy()
        for t in range(T):
            for j in range(k):
                if row[t, j] >= 0:
                    assert np.array_equal(qv[row[t, j]], want[t]) and np.array_equal(sv[row[t, j]], scale[t])
    assert tst.moe_status_query(plan) == tst.TST_OK


def test_dispatch_e4m3_of_rows_in_order_and_special_values():
    T, k, H = 12, 4, 384
    x = _normal(21, T * k, H).astype(np.float32)
    x[0] = 0
    x[1] *= 2.0 ** -110                                        # below the scale's floor
    x[2] *= 2.0 ** 100
    x[3, 5] = np.nan
    x[4, 200] = np.inf
    x[5, 380] = -np.inf
    x[6] = np.finfo(np.float32).max
    x[7, :128] = 2.0 ** -140                                   # subnormal
    plan = tst.moe_plan_create(T, 8, k)
    q = torch.zeros(T * k, H, dtype=torch.float8_e4m3fn, device="cuda")
    s = torch.zeros(T * k, 3, device="cuda")
    tst.moe_dispatch(plan, torch.from_numpy(x).cuda(), None, q, scales=s)
    qv, sv = _host(q), s.cpu().numpy()
    clean = [r for r in range(T * k) if r not in (3, 4, 5)]
    want, scale = moe.quantize(x[clean])
    assert np.array_equal(qv[clean], want) and np.array_equal(sv[clean], scale)
    # a tile with a NaN or an infinity cannot pass for a number; its neighbours are untouched
    assert np.isnan(sv[3, 0]) and np.isinf(sv[4, 1]) and np.isinf(sv[5, 2])
    assert np.isnan(qv[4, 200]) and np.isnan(qv[5, 380])
    assert np.isfinite(sv[3, 1:]).all() and np.isfinite(qv[3, 128:]).all() and np.isfinite(qv[4, :128]).all()


@pytest.mark.parametrize("T,k,H", [(1, 1, 1), (3, 2, 7), (17, 4, 1021), (40, 8, 4096), (19, 3, 520)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_dispatch_copies_rows(T, k, H, dtype):
    row, n, _ = _assign(T, k, 12, T + H, masked=True)
    x = _dev(_normal(500 + T, T, H), dtype)
    plan = tst.moe_plan_create(T, 12, k)
    for src in (x, _strided(x, 8), _strided(x, 1)):
        rows = torch.full((n + 2, H), float("nan"), dtype=x.dtype, device="cuda")
        tst.moe_dispatch(plan, src, torch.from_numpy(row).cuda(), rows)
        for t in range(T):
            for j in range(k):
                if row[t, j] >= 0:
                    assert torch.equal(rows[row[t, j]], x[t])
        assert rows[n:].isnan().all()                          # rows that no token names stay


@pytest.mark.parametrize("T,k,H", [(1, 1, 1), (2, 3, 8), (31, 4, 1021), (50, 8, 4096), (23, 2, 520), (5, 32, 264)])
@pytest.mark.parametrize("rows_type", ["f32", "bf16"])
@pytest.mark.parametrize("out_type", ["f32", "bf16"])
def test_combine_and_its_gradient_equal_the_oracle(T, k, H, rows_type, out_type):
    E = max(k, 9)
    row, n, weight = _assign(T, k, E, T + H, masked=T > 8)
    rows = _dev(_normal(600 + T, n + 1, H), rows_type)
    rows[n] = float("nan")                                     # a row that no token names
    d_row = torch.from_numpy(row).cuda()
    plan = tst.moe_plan_create(T, E, k)
    w = torch.from_numpy(weight).cuda()
    w[d_row < 0] = float("nan")                                # weights of no row are not read
    hw = np.where(row >= 0, weight, 0).astype(np.float64)
    for pad in (0, 8, 1):
        for wt, hwt in ((w, hw), (None, None)):
            out = _strided(torch.full((T, H), float("nan"), dtype=TYPES[out_type], device="cuda"), pad)
            tst.moe_combine(plan, rows, d_row, out, weight=wt)
            want, size = moe.combine(_host(rows), row, hwt)
            tol = (k + 1) * U * size + (half_ulp_bf16(want) if out_type == "bf16" else 0.0)
            assert (np.abs(_host(out) - want) <= tol).all()
        d_out = _strided(_dev(_normal(700 + T, T, H), out_type), pad)
        d_rows = torch.full_like(rows, float("nan"))
        d_weight = torch.full((T, k), float("nan"), device="cuda")
        tst.moe_combine_backward(plan, rows, d_row, w, d_out, d_rows, d_weight)
        want_r, want_w, size_w = moe.combine_backward(_host(rows), row, hw, _host(d_out))
        got = _host(d_rows)
        assert np.isnan(got[n]).all()
        tol = U * np.abs(want_r[:n]) + 2.0 ** -149 + (half_ulp_bf16(want_r[:n]) if rows_type == "bf16" else 0.0)
        assert (np.abs(got[:n] - want_r[:n]) <= tol).all()
        assert (np.abs(_host(d_weight) - want_w) <= (H / 256 + 24) * U * size_w).all()
    assert tst.moe_status_query(plan) == tst.TST_OK


def test_combine_without_weights_is_the_gradient_of_dispatch():
    # <dispatch(x), g> = <x, combine(g)> for small integers, exactly
    T, k, H = 29, 3, 264
    row, n, _ = _assign(T, k, 8, 5, masked=True)
    x = _dev(synthetic.draw("int:8", 31, T * H).reshape(T, H))
    g = _dev(synthetic.draw("int:8", 32, n * H).reshape(n, H))
    plan, d_row = tst.moe_plan_create(T, 8, k), torch.from_numpy(row).cuda()
    rows, back = torch.zeros(n, H, device="cuda"), torch.zeros(T, H, device="cuda")
    tst.moe_dispatch(plan, x, d_row, rows)
    tst.moe_combine(plan, g, d_row, back)
    assert (rows.double() * g.double()).sum().item() == (x.double() * back.double()).sum().item()


def test_rows_outside_the_matrix_are_skipped_and_reported():
    T, k, H = 4, 2, 128
    plan = tst.moe_plan_create(T, 8, k)
    row = torch.tensor([[0, 1], [2, 99], [-1, -5], [3, -1]], dtype=torch.int32, device="cuda")
    x = _dev(_normal(41, T, H))
    rows = torch.full((4, H), 7.0, device="cuda")
    tst.moe_dispatch(plan, x, row, rows)
    assert tst.moe_status_query(plan) == tst.TST_ERR_DEVICE_CHECK
    assert tst.moe_status_query(plan) == tst.TST_OK            # reported once
    assert torch.equal(rows, x[[0, 0, 1, 3]])
    out = torch.full((T, H), float("nan"), device="cuda")
    tst.moe_combine(plan, rows, row, out)
    assert tst.moe_status_query(plan) == tst.TST_ERR_DEVICE_CHECK
    assert torch.equal(out, torch.stack([rows[0] + rows[1], rows[2], torch.zeros_like(rows[0]), rows[3]]))
    d_rows, d_w = torch.zeros_like(rows), torch.zeros(T, k, device="cuda")
    tst.moe_combine_backward(plan, rows, row, torch.ones(T, k, device="cuda"), x, d_rows, d_w)
    assert tst.moe_status_query(plan) == tst.TST_ERR_DEVICE_CHECK
    assert d_w[2].tolist() == [0, 0] and d_w[1, 1].item() == 0 and torch.equal(d_rows[2], x[1])


def test_no_tokens_and_no_rows():
    plan = tst.moe_plan_create(8, 4, 2)
    none, row0 = torch.empty(0, 64, device="cuda"), torch.empty(0, 2, dtype=torch.int32, device="cuda")
    tst.moe_dispatch(plan, none, row0, none)
    tst.moe_combine(plan, none, row0, none)
    tst.moe_combine_backward(plan, none, row0, torch.empty(0, 2, device="cuda"), none, none, torch.empty(0, 2, device="cuda"))
    # tokens, but every one of them without rows
    row, out = torch.full((8, 2), -1, dtype=torch.int32, device="cuda"), torch.full((8, 64), float("nan"), device="cuda")
    tst.moe_dispatch(plan, torch.ones(8, 64, device="cuda"), row, none)
    tst.moe_combine(plan, none, row, out)
    d_w = torch.full((8, 2), float("nan"), device="cuda")
    tst.moe_combine_backward(plan, none, row, torch.ones(8, 2, device="cuda"), torch.ones(8, 64, device="cuda"), none, d_w)
    assert (out == 0).all() and (d_w == 0).all() and tst.moe_status_query(plan) == tst.TST_OK


def test_rows_past_two_gigabytes():
    # row offsets of more than 2^31 elements and 2^32 bytes: the last rows of a matrix of 4.3 GB
    n, H, T = (1 << 31) // 4096 + 8, 4096, 3
    plan = tst.moe_plan_create(T, 4, 2)
    row = torch.tensor([[n - 1, 0], [n - 3, n - 2], [1, -1]], dtype=torch.int32, device="cuda")
    x = _dev(_normal(51, T, H), "bf16")
    rows = torch.zeros(n, H, dtype=torch.bfloat16, device="cuda")
    tst.moe_dispatch(plan, x, row, rows)
    assert torch.equal(rows[n - 1], x[0]) and torch.equal(rows[n - 2], x[1]) and torch.equal(rows[1], x[2])
    out = torch.empty(T, H, device="cuda")
    tst.moe_combine(plan, rows, row, out)
    assert torch.equal(out[0], 2 * x[0].float()) and torch.equal(out[2], x[2].float())
    assert (rows[4:n - 4] == 0).all()


def test_refusals_of_the_binding():
    plan = tst.moe_plan_create(4, 8, 2)
    f = lambda *s: torch.zeros(*s, device="cuda")  # noqa: E731
    i = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    good = dict(logits=f(4, 8), expert=i(4, 2), weight=f(4, 2), row=i(4, 2), counts=i(8), totals=i(2), loss=f(1))
    for name, bad in (("logits", f(4, 7)), ("logits", f(4, 8).half()), ("logits", f(8, 4).t()), ("logits", f(32)),
                      ("expert", i(4, 3)), ("expert", f(4, 2)), ("weight", f(4, 2).double()), ("row", i(2, 4).t()[:, :1]),
                      ("counts", i(7)), ("totals", i(1)), ("loss", f(2)), ("logits", torch.zeros(4, 8))):
        with pytest.raises(ValueError):
            tst.moe_route(plan, **dict(good, **{name: bad}))
    with pytest.raises(ValueError):
        tst.moe_route(plan, **good, mask=i(4))
    with pytest.raises(tst.TstError) as e:                     # more tokens than the plan's
        tst.moe_route(plan, f(5, 8), i(5, 2), f(5, 2), i(5, 2), i(8), i(2), f(1))
    assert e.value.status == tst.TST_ERR_INVALID_ARG
    e4, s = torch.zeros(8, 24, dtype=torch.uint8, device="cuda"), f(8, 1)
    with pytest.raises(tst.TstError) as e:                     # e4m3 rows must be multiples of 16
        tst.moe_dispatch(plan, f(4, 24), i(4, 2), e4, scales=s)
    assert e.value.status == tst.TST_ERR_ALIGNMENT
    with pytest.raises(ValueError):                            # e4m3 rows without scales
        tst.moe_dispatch(plan, f(4, 32), i(4, 2), torch.zeros(8, 32, dtype=torch.uint8, device="cuda"))
    with pytest.raises(tst.TstError) as e:                     # a copy does not convert
        tst.moe_dispatch(plan, f(4, 24), i(4, 2), f(8, 24).bfloat16())
    assert e.value.status == tst.TST_ERR_UNSUPPORTED
    with pytest.raises(tst.TstError) as e:                     # rows in order need a row per token
        tst.moe_dispatch(plan, f(4, 24), None, f(3, 24))
    assert e.value.status == tst.TST_ERR_INVALID_ARG
    for bad in (dict(rows=f(8, 23)), dict(rows=f(24, 8).t()), dict(row=i(4, 1)), dict(weight=f(4, 3)), dict(out=f(4, 24).half())):
        with pytest.raises(ValueError):
            tst.moe_combine(plan, **dict(dict(rows=f(8, 24), row=i(4, 2), out=f(4, 24), weight=f(4, 2)), **bad))
    with pytest.raises(ValueError):
        tst.moe_combine_backward(plan, f(8, 24), i(4, 2), f(4, 2), f(4, 24), f(8, 24).bfloat16(), f(4, 2))
    plan.destroy()
    with pytest.raises(ValueError):
        tst.moe_route(plan, **good)
