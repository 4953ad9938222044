"""GPU parity of the int8 GEMM (gemm_int8_run) against exact integer sums.

With unit scales and FP32 output the result is the integer sum rounded once: equal bits.  With scales,
u = 2^-24: the sum's rounding, the row scale's product and the fused step with the channel's scale and the
bias are three roundings, the last of the result: 2.01 u |s ra cb| + 1.01 u |D|; BF16 output adds half a unit
in its last place."""
import numpy as np
import pytest
import torch

import tile_scheduled_tensor_gb300 as tst
from oracle import int8

from gemm_check import half_ulp_bf16

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def _dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def _operands(seed, M, N, K, parts=1, low=-127):
    rng = np.random.default_rng(seed)
    A, B = (rng.integers(low, 128, (n, K), dtype=np.int8) for n in (M, parts * N))
    ra, cb = (rng.uniform(0.25, 2.0, n).astype(np.float32) * np.float32(1e-3) for n in (M, parts * N))
    return A, B, ra, cb, rng.normal(size=parts * N).astype(np.float32)


def _run(plan, A, B, ra, cb, bias=None, group_rows=None, fill=float("nan")):
    D = torch.full((plan.M, plan.N), fill, dtype=torch.float32 if plan.out_dtype == tst.TST_OUT_F32 else torch.bfloat16, device="cuda")
    tst.gemm_int8_run(plan, _dev(A), _dev(B), D, _dev(ra), _dev(cb), bias=None if bias is None else _dev(bias),
                      group_rows=None if group_rows is None else _dev(np.asarray(group_rows, dtype=np.int32)))
    return D


def _check(D, want, size):
    got = D.float().cpu().numpy().astype(np.float64)
    tol = 2.01 * U * size + 1.01 * U * np.abs(want)
    if D.dtype == torch.bfloat16:
        tol = tol + 1.01 * half_ulp_bf16(want)
    assert (np.abs(got - want) <= tol).all(), float(np.max(np.abs(got - want) - tol))


# tokens on each side of the tile heights, ragged columns, K of less than a k-block, of whole folds and past them
SHAPES = [(1, 1, 16), (1, 128, 128), (2, 3, 48), (16, 130, 1024), (17, 129, 1040), (32, 64, 2048), (33, 257, 2064), (63, 500, 144),
          (64, 128, 4096), (65, 127, 1008), (128, 256, 1152), (129, 300, 4112), (256, 384, 512), (257, 1000, 8208), (700, 513, 3088)]


# every form: rows per tile, 1 without tiles.  num_sms 16: each CTA (or pair) takes many tiles
FORMS = [0, 1, 16, 32, 64, 128, 192]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("rows", FORMS)
@pytest.mark.parametrize("num_sms", [0, 16])
def test_sums_are_exact(M, N, K, rows, num_sms):
    A, B, _, _, _ = _operands(M + N + K, M, N, K, low=-128)
    plan = tst.gemm_int8_plan_create(M, N, K, out_dtype="f32", num_sms=num_sms, tile_rows=rows)
    assert rows in (0, plan.info.tile_rows)
    D = _run(plan, A, B, np.ones(M, np.float32), np.ones(N, np.float32))
    assert tst.gemm_int8_status_query(plan) == tst.TST_OK
    assert np.array_equal(D.cpu().numpy(), int8.sums(A, B).astype(np.float32))


@pytest.mark.parametrize("M,N,K", [(3, 5, 1024), (20, 140, 8192), (130, 260, 1040), (2, 3, 131056), (300, 260, 16384)])
@pytest.mark.parametrize("a,b", [(-128, -128), (-128, 127), (127, 127)])
@pytest.mark.parametrize("rows", FORMS)
def test_largest_magnitudes(M, N, K, a, b, rows):
    # every partial sum as large as it can be: 2^24 per accumulator, close to 2^31 over the longest K
    A, B = np.full((M, K), a, np.int8), np.full((N, K), b, np.int8)
    A[0, ::7], B[0, 1::5] = 1, -1   # and sums that are no multiple of a power of two
    plan = tst.gemm_int8_plan_create(M, N, K, out_dtype="f32", tile_rows=rows)
    D = _run(plan, A, B, np.ones(M, np.float32), np.ones(N, np.float32))
    assert np.array_equal(D.cpu().numpy(), int8.sums(A, B).astype(np.float32))


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_scales_bias_relu(M, N, K, out):
    A, B, ra, cb, bias = _operands(7 * M + N, M, N, K)
    for use_bias, relu, rows in ((False, False, 0), (True, True, 1), (True, True, 16), (True, False, 32), (True, True, 64), (True, False, 128),
                                 (True, True, 192)):
        plan = tst.gemm_int8_plan_create(M, N, K, out_dtype=out, has_bias=use_bias, relu=relu, tile_rows=rows)
        D = _run(plan, A, B, ra, cb, bias if use_bias else None)
        _check(D, *int8.gemm(A, B, ra, cb, bias if use_bias else None, relu))


GROUPS = [("one", 1, 5, 130, 272, [5]), ("long K", 3, 40, 384, 4112, [7, 0, 33]), ("empty first and last", 5, 40, 200, 1040, [0, 17, 0, 23, 0]),
          ("one row each", 60, 60, 96, 144, [1] * 60), ("uneven", 7, 333, 257, 2064, [1, 200, 0, 33, 64, 32, 3]),
          ("many", 300, 700, 130, 128, [(i * 7) % 5 for i in range(300)]), ("large", 3, 1500, 384, 1536, [129, 1000, 371]), ("large with rows to spare", 4, 1700, 300, 1040, [0, 600, 1, 500]),
          ("none", 4, 9, 64, 64, [0, 0, 0, 0])]


@pytest.mark.parametrize("name,G,M,N,K,rows", GROUPS, ids=[g[0] for g in GROUPS])
@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("tile", FORMS)
@pytest.mark.parametrize("num_sms", [0, 16])
def test_grouped(name, G, M, N, K, rows, out, tile, num_sms):
    A, B, ra, cb, bias = _operands(G + M, M, N, K, parts=G)
    plan = tst.gemm_int8_plan_create(M, N, K, groups=G, out_dtype=out, has_bias=True, num_sms=num_sms, tile_rows=tile)
    D = _run(plan, A, B, ra, cb, bias, rows, fill=-77.0)
    assert tst.gemm_int8_status_query(plan) == tst.TST_OK
    used = sum(rows)
    assert (D[used:] == -77.0).all()   # rows behind the last group's stay as they were
    want, size = int8.gemm(A[:used], B, ra[:used], cb, bias, False, rows)
    _check(D[:used], want, size)


@pytest.mark.parametrize("scale,rows", [(1, 0), (1, 1), (1, 16), (1, 32), (10, 64), (10, 128), (10, 192)])
def test_rows_past_the_matrix_are_reported(scale, rows):
    M = 100 * scale
    A, B, ra, cb, _ = _operands(3, M, 64, 128, parts=3)
    plan = tst.gemm_int8_plan_create(M, 64, 128, groups=3, out_dtype="f32", tile_rows=rows)
    D = _run(plan, A, B, ra, cb, None, [60 * scale, -4, 70 * scale])
    assert tst.gemm_int8_status_query(plan) == tst.TST_ERR_DEVICE_CHECK
    assert tst.gemm_int8_status_query(plan) == tst.TST_OK   # reported once
    want, size = int8.gemm(A, B, ra, cb, None, False, [60 * scale, 0, 40 * scale])
    _check(D, want, size)


def test_scales_that_are_not_numbers_stay_visible():
    A, B, ra, cb, bias = _operands(5, 4, 40, 64)
    ra[1], ra[2], cb[3] = np.nan, np.inf, np.nan
    D = _run(tst.gemm_int8_plan_create(4, 40, 64, out_dtype="f32", has_bias=True, relu=True), A, B, ra, cb, bias).cpu().numpy()
    assert np.isnan(D[1]).all() and np.isnan(D[:, 3]).all() and np.isfinite(D[0, 4:]).all()


@pytest.mark.parametrize("scale,tile", [(1, 0), (1, 1), (1, 16), (1, 32), (10, 64), (10, 128), (10, 192)])
def test_streams_and_graphs(scale, tile):
    # a plan on another stream, and captured: the replay reads what its inputs hold then
    G, M, N, K = 4, 90 * scale, 192, 1168
    A, B, ra, cb, bias = _operands(9, M, N, K, parts=G)
    A2 = _operands(10, M, N, K)[0]
    plan = tst.gemm_int8_plan_create(M, N, K, groups=G, out_dtype="f32", has_bias=True, tile_rows=tile)
    first, second = ([n * scale for n in rows] for rows in ([10, 0, 50, 30], [40, 41, 0, 9]))
    a, b, r, c, bs = (_dev(x) for x in (A, B, ra, cb, bias))
    rows = torch.tensor(first, dtype=torch.int32, device="cuda")
    D = torch.empty(M, N, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    tst.gemm_int8_run(plan, a, b, D, r, c, bias=bs, group_rows=rows, stream=s)
    s.synchronize()
    _check(D, *int8.gemm(A, B, ra, cb, bias, False, first))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tst.gemm_int8_run(plan, a, b, D, r, c, bias=bs, group_rows=rows)
    a.copy_(_dev(A2))
    rows.copy_(torch.tensor(second, dtype=torch.int32))
    D.fill_(float("nan"))
    graph.replay()
    torch.cuda.synchronize()
    _check(D, *int8.gemm(A2, B, ra, cb, bias, False, second))
    assert tst.gemm_int8_status_query(plan) == tst.TST_OK


def test_two_plans_at_once():
    # plans share nothing: two on two streams, many times
    jobs = []
    for i, (M, N, K) in enumerate([(12, 1024, 2048), (200, 640, 1040), (4000, 1300, 528)]):
        A, B, ra, cb, _ = _operands(20 + i, M, N, K)
        jobs.append((tst.gemm_int8_plan_create(M, N, K, out_dtype="f32"), [_dev(x) for x in (A, B)], torch.empty(M, N, device="cuda"),
                     [_dev(x) for x in (ra, cb)], torch.cuda.Stream(), int8.gemm(A, B, ra, cb)))
    torch.cuda.synchronize()
    for _ in range(20):
        for plan, (a, b), D, (r, c), s, _want in jobs:
            tst.gemm_int8_run(plan, a, b, D, r, c, stream=s)
    torch.cuda.synchronize()
    for _plan, _ab, D, _rc, _s, want in jobs:
        _check(D, *want)
