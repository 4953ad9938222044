"""Each form of the block-scaled kernels over its own paths: the tile heights and widths that a grouped
plan takes by its sizes, one scale of B per tile and one per column, the run after a wait that ran out,
row counts past the matrix, and dense plans of 128 x 256 tiles.  Bounds as in
test_grouped_block_scaled_gpu.py."""
import numpy as np
import pytest
import torch

import oracle
import synthetic
import tile_scheduled_tensor_gb300 as tst
from oracle import blockscale as BS

import test_grouped_block_scaled_gpu as base
from gemm_check import device_codes, half_ulp_bf16, host_values

pytestmark = pytest.mark.gpu

SHARED, PER_COL, SOME_COL = (1, 128, 128), (1, 128, 1), (1, 128, 48)
FEW, SOME, MANY = [1, 0, 3, 1, 2, 0, 5], [5, 0, 17, 1, 33, 2, 70], [60, 0, 131, 128, 1, 7, 90]
# rows, tiling, the form (bm, bn) that the plan takes, its options
FORMS = {
    "16 shared": (FEW, SHARED, (16, 128), {}), "16 per column": (FEW, PER_COL, (16, 128), {}), "16 of 48": (FEW, SOME_COL, (16, 128), {}),
    "32 shared": (SOME, SHARED, (32, 128), {}), "32 per column": (SOME, PER_COL, (32, 128), {}), "32 of 48": (SOME, SOME_COL, (32, 128), {}),
    "128 shared": (MANY, SHARED, (128, 128), {}), "128 per column": (MANY, PER_COL, (128, 128), {}),
    "256 wide": (MANY, SHARED, (128, 256), dict(bn=256)),
}


def _takes(rows, N, K, ab, form, **kw):
    info = tst.gemm_grouped_plan_create(len(rows), sum(rows), N, K, dtype="e4m3", ab_block=ab, host_only=True, num_sms=152, **kw).info
    assert (info.bm, info.bn) == form


@pytest.mark.parametrize("name", FORMS)
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_forms_exact(name, out):
    rows, ab, form, kw = FORMS[name]
    for N, K in ((264, 784), (130, 1168)):
        _takes(rows, N, K, ab, form, **kw)
        base._exact(rows, N, K, ab, out, alpha=0.5, bias=True, relu=out == "bf16", seed=N, **kw)


@pytest.mark.parametrize("name", FORMS)
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_forms_within_the_bound(name, out):
    rows, ab, form, kw = FORMS[name]
    N, K = 200, 1040
    _takes(rows, N, K, ab, form, **kw)
    got, z, size, st, _ = base._case(rows, N, K, ab, out=out, dist="normal", pow2=False, seed=6, **kw)
    assert st == tst.TST_OK
    tol = (4 * (K / 128 + 8) + 128) * 2.0 ** -24 * size + (half_ulp_bf16(z) if out == "bf16" else 0.0)
    assert (np.abs(got - z) <= tol).all(), float((np.abs(got - z) / tol).max())


@pytest.mark.parametrize("name", FORMS)
def test_forms_recover_after_a_missing_load(name):
    # the producer skips one load (a host-set flag): the bounded wait runs out and the run ends with
    # TST_ERR_TIMEOUT, which base._case asserts; the next run is right
    rows, ab, form, kw = FORMS[name]
    N, K = 300, 1040
    _takes(rows, N, K, ab, form, **kw)
    got, z, _, st, _ = base._case(rows, N, K, ab, seed=4, fault=True, **kw)
    assert st == tst.TST_OK and np.array_equal(got, z)


@pytest.mark.parametrize("name", FORMS)
def test_forms_report_more_rows_than_the_matrix(name):
    # the last two groups' counts pass the matrix, the last one starts past it: what fits is right
    rows, ab, form, kw = FORMS[name]
    N, K = 264, 272
    rows = rows + [0]
    _takes(rows, N, K, ab, form, **kw)
    run = rows[:-2] + [rows[-2] + 41, 6]
    got, z, _, st, _ = base._case(rows, N, K, ab, run=run, seed=7, **kw)
    assert st == tst.TST_ERR_DEVICE_CHECK
    assert np.array_equal(got, z)


@pytest.mark.parametrize("schedule,mapping", [("static", ("linear_nfast", 1)), ("persistent", ("grouped_n", 2)), ("persistent", ("morton", 1))])
@pytest.mark.parametrize("M,N,K", [(1, 1, 16), (128, 256, 128), (300, 520, 400), (257, 300, 1040), (130, 1416, 2064)])
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_dense_wide_tiles_exact(M, N, K, schedule, mapping, out):
    A = synthetic.e4m3_bytes(synthetic.draw("int:4", 8100 + M, M * K).reshape(M, K).astype(np.float32))
    B = synthetic.e4m3_bytes(synthetic.draw("int:4", 8200 + N, N * K).reshape(N, K).astype(np.float32))
    sA, sB = base._scales(8300 + M, (M, -(-K // 128)), True), base._scales(8400 + N, (-(-N // 128), -(-K // 128)), True)
    bias = synthetic.draw("int:4", 8500 + N, N).astype(np.float32)
    plan = tst.gemm_plan_create(M, N, K, dtype="e4m3", mapping=mapping, schedule=schedule, out_dtype=out, alpha=0.5, has_bias=True,
                                relu=out == "bf16", ab_block=SHARED, bn=256)
    assert (plan.info.bm, plan.info.bn) == (128, 256)
    D = torch.full((M, N), float("nan"), dtype=torch.float32 if out == "f32" else torch.bfloat16, device="cuda")
    tst.gemm_run(plan, device_codes(A), device_codes(B), D, bias=torch.from_numpy(bias).cuda(), a_block_scales=torch.from_numpy(sA).cuda(),
                 b_block_scales=torch.from_numpy(sB).cuda())
    st, word = tst.gemm_status_query(plan)
    assert st == tst.TST_OK, hex(word)
    z = 0.5 * BS.gemm_block_scaled(oracle.decode(A, "e4m3"), oracle.decode(B, "e4m3"), sA, sB, (1, 128), block_rows_b=128) + bias.astype(np.float64)
    if out == "bf16":
        z = np.maximum(z, 0)
    want = z if out == "f32" else oracle.decode(oracle.round_bf16(z), "bf16")
    got = host_values(D)
    assert np.array_equal(got, want), np.argwhere(got != want)[:5]
