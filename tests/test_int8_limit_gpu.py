"""A wait of the int8 GEMM that runs out: plans whose limit is shorter than the work report it and end, with nothing in
flight, and whatever runs next is right."""
import pytest
import torch

import tile_scheduled_tensor_gb300 as tst

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def operands():
    M, N, K = 4096, 2048, 4096
    gen = torch.Generator(device="cuda").manual_seed(7)
    A, B = (torch.randint(-128, 128, (n, K), dtype=torch.int8, device="cuda", generator=gen) for n in (M, N))
    # FP32 adds 1024 products of int8 exactly
    want = sum((A[:, c:c + 1024].float() @ B[:, c:c + 1024].float().t()).int() for c in range(0, K, 1024)).float()
    return A, B, torch.ones(M, device="cuda"), torch.ones(N, device="cuda"), want


@pytest.mark.parametrize("rows", [16, 32, 64, 128, 192])
@pytest.mark.parametrize("num_sms", [0, 16])
def test_a_limit_that_runs_out(operands, rows, num_sms):
    A, B, ra, cb, want = operands
    M, N, K = A.shape[0], B.shape[0], A.shape[1]
    new = lambda **kw: tst.gemm_int8_plan_create(M, N, K, out_dtype="f32", tile_rows=rows, num_sms=num_sms, **kw)  # noqa: E731
    good = new()
    # 1 ns: the copy of A to FP16 alone takes microseconds, in which the MMA issuers wait for it.  The others run out, or not,
    # somewhere on the way.
    for limit in (1, 3000, 10000, 30000):
        plan = new(timeout_ns=limit)
        for _ in range(4):
            D = torch.full((M, N), float("nan"), device="cuda")
            tst.gemm_int8_run(plan, A, B, D, ra, cb)
            status = tst.gemm_int8_status_query(plan)
            assert status in ((tst.TST_ERR_TIMEOUT,) if limit == 1 else (tst.TST_OK, tst.TST_ERR_TIMEOUT))
            assert status != tst.TST_OK or torch.equal(D, want)
            assert tst.gemm_int8_status_query(plan) == tst.TST_OK   # reported once
        D.fill_(float("nan"))
        tst.gemm_int8_run(good, A, B, D, ra, cb)
        assert tst.gemm_int8_status_query(good) == tst.TST_OK and torch.equal(D, want)


def test_groups_whose_limit_runs_out():
    G, M, N, K = 6, 3000, 512, 2048
    gen = torch.Generator(device="cuda").manual_seed(8)
    A, B = (torch.randint(-128, 128, (n, K), dtype=torch.int8, device="cuda", generator=gen) for n in (M, G * N))
    counts = [700, 0, 900, 1, 1000, 299]
    rows = torch.tensor(counts, dtype=torch.int32, device="cuda")
    group = torch.repeat_interleave(torch.arange(G, device="cuda"), rows.long(), output_size=sum(counts))
    want = torch.empty(sum(counts), N, device="cuda")
    for g in range(G):
        a, b = A[:sum(counts)][group == g], B[g * N:(g + 1) * N]
        want[group == g] = sum((a[:, c:c + 1024].float() @ b[:, c:c + 1024].float().t()).int() for c in range(0, K, 1024)).float()
    ra, cb = torch.ones(M, device="cuda"), torch.ones(G * N, device="cuda")
    for tile in (16, 32, 64, 128, 192):
        for limit in (1, 5000, 0):
            plan = tst.gemm_int8_plan_create(M, N, K, groups=G, out_dtype="f32", tile_rows=tile, timeout_ns=limit)
            D = torch.full((M, N), -5.0, device="cuda")
            tst.gemm_int8_run(plan, A, B, D, ra, cb, group_rows=rows)
            status = tst.gemm_int8_status_query(plan)
            assert status in (tst.TST_OK, tst.TST_ERR_TIMEOUT) and (limit or status == tst.TST_OK)
            assert status != tst.TST_OK or torch.equal(D[:sum(counts)], want)
            assert (D[sum(counts):] == -5.0).all()
