"""Softmax scores without a bias are compared as e^(l - max), before the division that all share: one rule on every path,
whether a row's experts fit the list of those in reach or not."""
import numpy as np
import pytest
import torch

import tile_scheduled_tensor_gb300 as tst

from test_score_gpu import _dev, _route

pytestmark = pytest.mark.gpu


# 1 and 1 - 2^-53, which division by 84, 126 or 252 makes one number and by 20 or 100 does not; up to 32 are listed
@pytest.mark.parametrize("E", [20, 27, 84, 100, 126, 252])
@pytest.mark.parametrize("T", [1, 200, 9800])
def test_scores_a_step_of_fp64_apart(E, T):
    k, low = 4, 5
    l = np.zeros((T, E))
    l[:, :low] = -2.0 ** -53                      # the lower experts' scores are less by one step
    if T > 1:
        l[1] = 0.0                                # a tie of all
    rank = np.argsort(-np.exp(l), axis=1, kind="stable")[:, :k]
    assert rank[0].tolist() == [5, 6, 7, 8]
    plan = tst.moe_plan_create(T, E, k, score="softmax")
    o = _route(plan, _dev(l))
    assert np.array_equal(o["expert"].cpu().numpy(), rank)
    # a bias of zeros: the values are s + 0, so s as divided
    c = np.exp(l) / np.exp(l).sum(axis=1, keepdims=True)
    want = np.argsort(-c, axis=1, kind="stable")[:, :k]
    o = _route(plan, _dev(l), torch.zeros(E, device="cuda"))
    assert np.array_equal(o["expert"].cpu().numpy(), want)


def test_a_missing_number_makes_all_of_its_row_equal():
    # softmax of a row with a NaN or +inf is NaN, which counts as +inf for every open expert
    l = np.zeros((3, 40))
    l[0, 7], l[1, 9], l[2, 11], l[2, 3] = np.nan, np.inf, np.nan, -np.inf
    l[:, 20:] = 5.0
    o = _route(tst.moe_plan_create(3, 40, 5, score="softmax"), _dev(l))
    assert o["expert"].tolist() == [[0, 1, 2, 3, 4], [0, 1, 2, 3, 4], [0, 1, 2, 4, 5]]
