"""GPU parity of the grouped GEMM with block-scaled FP8 operands (gemm_grouped_plan_create with
ab_block) against the oracle's gemm_block_scaled, group by group: A's scales belong to the rows of
the whole A, each group has its own B and its own scales of B.

Exact with small integers and power-of-two scales; random e4m3 codes with scales that are not
powers of two lie within K / 128 + 8 units roundoff per 128-element partial's fold of FP32, taken as
4 (K / 128 + 8) 2^-24 of sum |a sA| |b sB| for the folds and the tensor core's sums of 128 exact
products 128 2^-24 of it, and half a unit in the last place of a BF16 result."""
import numpy as np
import pytest
import torch

import oracle
import synthetic
import tile_scheduled_tensor_gb300 as tst
from oracle import blockscale as BS

from gemm_check import device_codes, half_ulp_bf16, host_values

pytestmark = pytest.mark.gpu


def _scales(seed, shape, pow2):
    n = int(np.prod(shape))
    if pow2:
        e = (synthetic.splitmix64(seed, n) % np.uint64(7)).astype(np.int64) - 3
        return (2.0 ** e).reshape(shape).astype(np.float32)
    return (0.5 + 1.5 * synthetic.uniform01(seed, n)).reshape(shape).astype(np.float32)


def _case(rows, N, K, ab, *, out="f32", dtype="e4m3", dist="int:4", pow2=True, alpha=1.0, bias=False, relu=False, spare=0,
          seed=0, run=None, fault=False, **plan_kw):
    """(got, z, absolute sums) of the groups' rows; `spare` rows of capacity past them."""
    br, bk, br_b = (tuple(ab) + (ab[0],))[:3]
    M, G = sum(rows) + spare, len(rows)
    fa, fb = synthetic.operand_types(dtype)
    enc = {"e4m3": synthetic.e4m3_bytes, "e5m2": synthetic.e5m2_bytes}
    A = enc[fa](synthetic.draw(dist, 7100 + seed, M * K).reshape(M, K).astype(np.float32))
    B = enc[fb](synthetic.draw(dist, 7200 + seed, G * N * K).reshape(G * N, K).astype(np.float32))
    sA = _scales(7300 + seed, (-(-M // br), -(-K // bk)), pow2)
    sB = _scales(7400 + seed, (G, -(-N // br_b), -(-K // bk)), pow2)
    bv = synthetic.draw("int:4", 7500 + seed, N).astype(np.float32) if bias else None
    plan = tst.gemm_grouped_plan_create(G, M, N, K, dtype=dtype, out_dtype=out, alpha=alpha, has_bias=bias, relu=relu, ab_block=ab,
                                        **plan_kw)
    D = torch.full((M, N), float("nan"), dtype=torch.float32 if out == "f32" else torch.bfloat16, device="cuda")
    counts = torch.tensor(rows if run is None else run, dtype=torch.int32, device="cuda")
    dA, dB, d_bias = device_codes(A), device_codes(B), None if bv is None else torch.from_numpy(bv).cuda()
    scales = dict(a_block_scales=torch.from_numpy(sA).cuda(), b_block_scales=torch.from_numpy(sB).cuda())
    if fault:
        tst.gemm_plan_set_debug(plan, tst.TST_DEBUG_FAULT_SKIP_LOAD, None, 0, timeout_ns=20_000_000)
        tst.gemm_grouped_run(plan, counts, dA, dB, D, bias=d_bias, **scales)
        assert tst.gemm_status_query(plan)[0] == tst.TST_ERR_TIMEOUT
        tst.gemm_plan_set_debug(plan, 0, None, 0)
    tst.gemm_grouped_run(plan, counts, dA, dB, D, bias=d_bias, **scales)
    st, word = tst.gemm_status_query(plan)
    a, b = oracle.decode(A, fa), oracle.decode(B, fb)
    z, size = np.zeros((sum(rows), N)), np.zeros((sum(rows), N))
    at = 0
    for g, r in enumerate(rows):
        if r:
            part, bg = np.arange(at, at + r), b[g * N:(g + 1) * N]
            z[part] = alpha * BS.gemm_block_scaled(a, bg, sA, sB[g], (br, bk), rows=part, block_rows_b=br_b)
            size[part] = abs(alpha) * BS.gemm_block_scaled(np.abs(a), np.abs(bg), sA, sB[g], (br, bk), rows=part,
                                                           block_rows_b=br_b)
        at += r
    if bias:
        z += bv.astype(np.float64)[None, :]
    if relu:
        z = np.maximum(z, 0)
    return host_values(D), z, size, st, word


def _exact(rows, N, K, ab, out="f32", **kw):
    got, z, _, st, word = _case(rows, N, K, ab, out=out, **kw)
    assert st == tst.TST_OK, (tst.gemm_status_string(st), hex(word))
    n = sum(rows)
    assert np.abs(z).max(initial=0) < 2 ** 22
    want = z if out == "f32" else oracle.decode(oracle.round_bf16(z), "bf16")
    assert np.array_equal(got[:n], want), np.argwhere(got[:n] != want)[:5]
    assert np.isnan(got[n:]).all()                # rows past the groups' are left alone


@pytest.mark.parametrize("rows", [[1], [0, 1, 0], [1] * 9, [3, 0, 130, 128, 1, 0, 17], [127, 129, 256], [0, 0, 500], [33, 31, 64, 65]])
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_groups_of_every_size_exact(rows, out):
    _exact(rows, 328, 1040, (1, 128, 128), out, spare=5, alpha=0.5, bias=True, relu=out == "bf16", seed=len(rows))


@pytest.mark.parametrize("N,K", [(1, 16), (8, 128), (127, 144), (128, 256), (130, 272), (256, 2064), (1416, 128)])
def test_odd_n_and_k_exact(N, K):
    for rows in ([2, 0, 5, 1], [140, 3]):
        for out in ("f32", "bf16"):
            _exact(rows, N, K, (1, 128, 128), out, seed=N + K)


@pytest.mark.parametrize("ab", [(1, 32), (32, 32), (1, 64, 128), (128, 128), (1, 128, 1), (1, 128, 48)])
def test_other_tilings_exact(ab):
    # A's scale tiles are those of the whole A, also where a group starts inside one
    _exact([45, 0, 1, 200, 18], 200, 528, ab, seed=ab[0] + ab[1])


@pytest.mark.parametrize("kw", [dict(num_ctas=3), dict(stages=2, num_ctas=5), dict(mapping=("grouped_n", 2)),
                                dict(mapping=("linear_mfast", 1)), dict(dtype="e5m2_e4m3")])
def test_schedules_and_formats_exact(kw):
    _exact([45, 0, 1, 300, 18, 2, 129], 520, 640, (1, 128, 128), seed=3, **kw)


def test_many_groups_exact():
    # more groups than a warp searches at once, most of them empty
    rows = [int(v) for v in (synthetic.splitmix64(77, 150) % np.uint64(4))]
    rows[10:60] = [0] * 50
    _exact(rows, 136, 256, (1, 128, 128), seed=8)


def test_more_groups_than_the_table_exact():
    rows = [int(v) for v in (synthetic.splitmix64(78, 600) % np.uint64(3))]
    _exact(rows, 40, 144, (1, 128, 128), seed=9)


# capacities that make the plan take each tile height
@pytest.mark.parametrize("spare", [0, 100, 400, 2000])
@pytest.mark.parametrize("ab", [(1, 128, 128), (1, 128, 1), (128, 128)])
def test_every_tile_height_exact(spare, ab):
    _exact([5, 0, 17, 1, 33, 2, 70], 264, 784, ab, seed=spare + ab[0], spare=spare)


# wide tiles: asked for, ragged in N and K, with short last row tiles, odd k-block counts and two stages
@pytest.mark.parametrize("N,K,kw", [(256, 128, {}), (300, 400, {}), (1416, 2064, {}), (520, 640, dict(stages=2, num_ctas=5)),
                                    (100, 272, {}), (770, 1152, dict(num_ctas=2))])
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_wide_tiles_exact(N, K, kw, out):
    _exact([300, 0, 1, 130, 33, 256], N, K, (1, 128, 128), out, bn=256, alpha=0.5, bias=True, relu=out == "bf16", seed=N, spare=3,
           **kw)


def test_plans_choose_wide_tiles_for_many_rows():
    big = tst.gemm_grouped_plan_create(16, 16384, 4096, 512, dtype="e4m3", ab_block=(1, 128, 128))
    assert tst.gemm_plan_get_info(big).bn == 256
    got, z, size, st, _ = _case([1500, 0, 900, 1696], 4096, 384, (1, 128, 128), out="bf16", seed=2)
    assert st == tst.TST_OK and np.array_equal(got, oracle.decode(oracle.round_bf16(z), "bf16"))


@pytest.mark.parametrize("rows,cap", [([3, 0, 5, 1], 9), ([40, 0, 20, 61], 121), ([300, 1, 0, 513], 900)])
def test_the_device_walks_the_enumerated_items(rows, cap):
    N, K, G = 520, 256, len(rows)
    plan = tst.gemm_grouped_plan_create(G, cap, N, K, dtype="e4m3", ab_block=(1, 128, 128), num_ctas=7)
    info = tst.gemm_plan_get_info(plan)
    trace = torch.full((info.grid * info.max_items_per_cta * 8,), -1, dtype=torch.int32, device="cuda")
    tst.gemm_plan_set_debug(plan, tst.TST_DEBUG_TRACE, trace, trace.numel())
    z = lambda *s: torch.zeros(*s, dtype=torch.uint8, device="cuda")  # noqa: E731
    tst.gemm_grouped_run(plan, torch.tensor(rows, dtype=torch.int32, device="cuda"), z(cap, K), z(G * N, K),
                         torch.empty(cap, N, dtype=torch.bfloat16, device="cuda"), a_block_scales=torch.zeros(cap, 2, device="cuda"),
                         b_block_scales=torch.zeros(G, 5, 2, device="cuda"))
    assert tst.gemm_status_query(plan)[0] == tst.TST_OK
    rec = trace.cpu().numpy().reshape(info.grid, info.max_items_per_cta, 8)
    for u in range(info.grid):
        want = tst.gemm_grouped_work_items(plan, rows, u)
        got = [tuple(r[2:8]) for r in rec[u] if r[0] >= 0]
        assert got == want, u


@pytest.mark.parametrize("cap", [20, 2000])
def test_a_missing_load_times_out_and_the_plan_recovers(cap):
    # the producer skips one load (a host-set flag): the issuer's bounded wait runs out, the run
    # ends with TST_ERR_TIMEOUT, and the next one is right
    rows, N, K = [4, 0, 9], 200, 512
    got, z, _, st, _ = _case(rows, N, K, (1, 128, 128), spare=cap - 13, seed=4, fault=True)
    assert st == tst.TST_OK and np.array_equal(got[:13], z)


def test_no_rows_at_all():
    got, _, _, st, _ = _case([0, 0, 0], 136, 256, (1, 128, 128), spare=64)
    assert st == tst.TST_OK and np.isnan(got).all()


@pytest.mark.parametrize("rows,N,K", [([5, 1, 0, 20, 9], 512, 2048), ([300, 77], 264, 1040)])
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_random_values_within_the_bound(rows, N, K, out):
    got, z, size, st, _ = _case(rows, N, K, (1, 128, 128), out=out, dist="normal", pow2=False, seed=5)
    assert st == tst.TST_OK
    tol = (4 * (K / 128 + 8) + 128) * 2.0 ** -24 * size + (half_ulp_bf16(z) if out == "bf16" else 0.0)
    assert (np.abs(got - z) <= tol).all(), float((np.abs(got - z) / tol).max())


def test_more_rows_than_the_matrix_is_reported():
    # the counts add up to more rows than A has: what fits is right, and the run says so
    got, z, _, st, _ = _case([40, 60], 136, 256, (1, 128, 128), run=[40, 90], seed=6)
    assert st == tst.TST_ERR_DEVICE_CHECK
    assert np.array_equal(got, z)


def test_scales_are_required():
    plan = tst.gemm_grouped_plan_create(2, 64, 128, 128, dtype="e4m3", ab_block=(1, 128, 128))
    t = torch.zeros(64 * 128 * 4, dtype=torch.uint8, device="cuda")
    for scales in (dict(), dict(a_block_scales=t), dict(b_block_scales=t)):
        with pytest.raises(tst.TstError) as e:
            tst.gemm_grouped_run(plan, torch.zeros(2, dtype=torch.int32, device="cuda"), t, t, t, **scales)
        assert e.value.status == tst.TST_ERR_INVALID_ARG
