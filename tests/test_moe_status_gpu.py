"""The status word of a mixture-of-experts plan: work on the default stream does not clear what a run on
another stream recorded."""
import pytest
import torch

import tile_scheduled_tensor_gb300 as tst

pytestmark = pytest.mark.gpu


def _bad_dispatch(plan, stream, x, row, rows):
    with torch.cuda.stream(stream):
        tst.moe_dispatch(plan, x, row, rows)


def test_a_record_survives_a_busy_default_stream():
    x = torch.ones(2, 64, device="cuda")
    row = torch.tensor([[0], [9]], dtype=torch.int32, device="cuda")   # row 9 of a matrix of two: skipped and recorded
    rows = torch.zeros(2, 64, device="cuda")
    warm = tst.moe_plan_create(2, 4, 1)
    side = torch.cuda.Stream()
    _bad_dispatch(warm, side, x, row, rows)
    assert tst.moe_status_query(warm) == tst.TST_ERR_DEVICE_CHECK
    assert tst.moe_status_query(warm) == tst.TST_OK
    torch.cuda.synchronize()
    torch.cuda._sleep(400_000_000)   # cycles: some 0.2 s of a kernel that does nothing, on the default stream
    plan = tst.moe_plan_create(2, 4, 1)
    _bad_dispatch(plan, side, x, row, rows)
    side.synchronize()
    busy = not torch.cuda.default_stream().query()
    torch.cuda.synchronize()
    assert tst.moe_status_query(plan) == tst.TST_ERR_DEVICE_CHECK
    assert tst.moe_status_query(plan) == tst.TST_OK
    assert busy, "the default stream was idle by then: nothing was shown"
