"""Routing and its gradient for finite logits of every magnitude, against the FP64 oracle: rows of
equal logits (a masked row's fill value among them), rows whose logits lie a few units in the last
place apart, and rows with one logit far above the rest.  Tolerances as in test_moe_gpu.py, whose
derivation holds for any finite logits: the distances to the row's largest logit count, not the logits."""
import numpy as np
import pytest
import torch

import tile_scheduled_tensor_gb300 as tst
from oracle import moe

from test_moe_gpu import _check_grad, _check_route, _dev, _host, _normal, _route

pytestmark = pytest.mark.gpu

# tops on both sides of powers of two, none of them a power of two, to the largest finite value
TOPS = [3.0, 1.04e6, 1.06e6, 1.7e7, 4.1e8, 1e9, 1.07e9, 2.2e9, 3e9, 5e9, 1e10, 1.1e12, 1e20, 6.3e29, 1e30, 1.3e30, 3e38]


def _rows(T, E, seed):
    """T rows: an ordinary one now and then, the others from TOPS, either sign, of the three kinds in turn."""
    l = _normal(seed, T, E)
    steps = np.random.default_rng(seed)
    for t in range(T):
        if t % 7 == 6:
            continue
        top = np.float32(TOPS[t % len(TOPS)] * (1 if (t // 3) % 2 else -1))
        kind = t % 3
        if kind == 0:
            l[t] = top
        elif kind == 1:   # exact in FP32: the row's distances are what the oracle sees
            l[t] = top - steps.integers(0, 40, E) * np.spacing(np.abs(top))
        else:
            l[t, steps.integers(0, E)] = abs(top)
    return l


# both kernels of routing and of its gradient at each of their widths, few and many tokens
SHAPES = [(120, 1, 1), (120, 6, 2), (121, 16, 4), (119, 32, 32), (120, 33, 6), (122, 64, 8), (120, 129, 7), (90, 256, 8), (88, 300, 32),
          (60, 1000, 9), (5200, 60, 4)]


@pytest.mark.parametrize("T,E,k", SHAPES)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_finite_logits_give_the_softmax(T, E, k, dtype):
    logits = _dev(_rows(T, E, 900 + E), dtype)
    l = _host(logits)
    assert np.isfinite(l).all()
    for normalize in (True, False):
        plan = tst.moe_plan_create(T, E, k, normalize=normalize, balance_coef=0.5)
        o = _route(plan, logits)
        want = moe.route(l, k, normalize, 0.5)
        assert np.isfinite(want["loss"])
        _check_route(o, want, l, normalize)


@pytest.mark.parametrize("T,E,k", SHAPES[:-1])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_finite_logits_give_finite_gradients(T, E, k, dtype):
    logits = _dev(_rows(T, E, 950 + E), dtype)
    l = _host(logits)
    dw = _dev(_normal(960 + E, T, k))
    for normalize in (True, False):
        plan = tst.moe_plan_create(T, E, k, normalize=normalize, balance_coef=0.5)
        o = _route(plan, logits)
        r = moe.route(l, k, normalize, 0.5)
        d = torch.full_like(logits, float("nan"))
        tst.moe_route_backward(plan, logits, o["expert"], o["counts"], o["totals"], d, d_weight=dw,
                               d_loss=torch.tensor([0.75], device="cuda"))
        assert d.isfinite().all()
        _check_grad(d, l, _host(dw), 0.75, r, normalize, 0.5, None, dtype)


@pytest.mark.parametrize("E", [20, 64])
@pytest.mark.parametrize("fill", [-1e9, -1e10, -1e30])
def test_one_filled_row_leaves_the_batch_its_loss(E, fill):
    # a padding row filled with a finite mask value, on a token that no mask byte closes
    T, k = 40, 4
    l = _normal(970, T, E)
    l[17] = fill
    logits = _dev(l)
    plan = tst.moe_plan_create(T, E, k)
    o = _route(plan, logits)
    assert np.isfinite(o["loss"].item())
    assert torch.allclose(o["weight"][17], torch.full((k,), 1.0 / k, device="cuda"))
    _check_route(o, moe.route(_host(logits), k, True, 0.01), _host(logits), True)
