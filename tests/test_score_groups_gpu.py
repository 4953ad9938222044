"""Expert groups whose values are sums of two: scores with biases far larger than the scores' differences, of both signs
and up to the type's lowest value.  Choices, counts and rows equal the FP64 oracle's.

Rows in which the last group kept and the first one dropped are closer than FP64 itself tells are left out: a value is within
3 u' of the formula's (u' = 2^-53, in units of the largest |c|), a sum of two within 8, so 2^-48 = 32 u' tells."""
import numpy as np
import pytest
import torch

import tile_scheduled_tensor_gb300 as tst
from oracle import moe

from test_score_gpu import _check, _dev, _host, _route

pytestmark = pytest.mark.gpu
LOWEST = float(np.finfo(np.float32).min)


def _apart(l, bias, sigmoid, G, g):
    """Rows whose kept groups do not hang on FP64's roundings."""
    c = np.stack([moe.scores(r, sigmoid) for r in l]) + bias.astype(np.float64)
    value = np.sort(c.reshape(len(l), G, -1), axis=2)[:, :, -2:].sum(axis=2)
    value = -np.sort(-value, axis=1)
    return (np.ones(len(l)) if g == G else value[:, g - 1] - value[:, g] > 2.0 ** -48 * np.abs(c).max()).astype(np.uint8)


def _compare(l, bias, score, k, G, g, best, mask=None):
    T, E = l.shape
    logits = _dev(l)
    l, sigmoid = _host(logits), score == "sigmoid"
    plan = tst.moe_plan_create(T, E, k, normalize=False, balance_coef=0.5, score=score, groups=G, top_groups=g, group_best=best)
    want = moe.route_scored(l, k, sigmoid, bias, G, g, best, False, 1.0, 0.5, mask=mask)
    _check(_route(plan, logits, _dev(bias), None if mask is None else torch.from_numpy(mask).cuda()), want, l)
    return want


# the smaller calls run in blocks of 32 rows, 9800 in larger ones; groups of 2 to 32 experts
@pytest.mark.parametrize("T,E,k,G,g,size,spread", [(3000, 4, 2, 2, 1, 1000.0, 1e-3), (9800, 4, 1, 2, 1, 1000.0, 1e-3), (2000, 16, 4, 4, 2, 128.0, 1.0),
                                                   (1000, 1024, 16, 32, 16, 64.0, 1.0), (2000, 96, 6, 3, 1, 1000.0, 0.01)])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_group_values_of_opposite_signs(T, E, k, G, g, size, spread, score):
    # one expert of each group is drawn in and the others are held off, as far: the sums are of the scores' size
    rng = np.random.default_rng(E + T)
    l = (spread * rng.normal(size=(T, E))).astype(np.float32).astype(np.float64)
    bias = np.full(E, -size, np.float32)
    bias[np.arange(G) * (E // G) + rng.integers(0, E // G, G)] = size
    mask = _apart(l, bias, score == "sigmoid", G, g)
    assert mask.mean() > 0.99
    _compare(l, bias, score, k, G, g, 2, mask)


def test_a_group_of_opposite_signs_beside_one_without_biases():
    l = np.array([[8e-5, 0.0, 2e-5, 0.0], [2e-5, 0.0, 8e-5, 0.0], [0.0, 8e-5, 0.0, 2e-5]])
    want = _compare(l, np.array([1000.0, -1000.0, 0.0, 0.0], np.float32), "sigmoid", 1, 2, 1, 2)
    assert want["expert"][:, 0].tolist() == [0, 2, 0]


def _lowest(E, *off, value=LOWEST):
    bias = np.zeros(E, np.float32)
    for part in off:
        bias[part] = value
    return bias


# the second group held off: its experts come last; two of three groups; all; one expert of each group left; a part of one
LOW = [(8, 6, 2, 2, _lowest(8, slice(4, 8))), (8, 8, 2, 2, _lowest(8, slice(0, 4))), (12, 5, 3, 2, _lowest(12, slice(0, 8))),
       (12, 4, 3, 1, _lowest(12, slice(0, 12))), (64, 16, 8, 4, _lowest(64, *[slice(i + 1, i + 8) for i in range(0, 64, 8)])),
       (256, 20, 8, 4, _lowest(256, slice(0, 160), slice(170, 255))), (256, 8, 8, 4, _lowest(256, slice(0, 3), slice(100, 108)))]


@pytest.mark.parametrize("E,k,G,g,bias", LOW, ids=[f"{c[0]}-{i}" for i, c in enumerate(LOW)])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("best", [1, 2])
@pytest.mark.parametrize("T", [40, 5000])
def test_biases_of_the_lowest_value(E, k, G, g, bias, score, best, T):
    # a group's sum of two is beyond FP32, its experts are not closed
    want = _compare(np.random.default_rng(E + G).normal(size=(T, E)), bias, score, k, G, g, best)
    assert (want["expert"] >= 0).all()


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_sums_beyond_fp32_keep_their_order(score):
    # -6e38, -4e38, -6.8e38 and -5e38 for the groups; and the same above zero
    size = np.repeat(np.array([3e38, 2e38, 3.4e38, 2.5e38]), 4)
    l = np.random.default_rng(3).normal(size=(50, 16))
    for bias in ((-size).astype(np.float32), size.astype(np.float32)):
        for g in (1, 2, 3):
            want = _compare(l, bias, score, 4, 4, g, 2)
            first = 4 if bias[0] < 0 else 8
            assert (want["expert"] // 4 == first // 4).all()
