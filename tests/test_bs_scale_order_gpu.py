"""A block's factor is the FP32 product of its two scales, in every form of the block-scaled kernels: scales
far from one whose product is ordinary give the ordinary result, exactly (small integers, powers of two)."""
import numpy as np
import pytest

import tile_scheduled_tensor_gb300 as tst

import test_grouped_block_scaled_gpu as base
from test_grouped_bs_forms_gpu import FORMS

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("name", FORMS)
@pytest.mark.parametrize("power_a,power_b", [(-100, 124), (124, -100), (-120, 118)])
def test_factor_is_the_product_of_the_scales(name, power_a, power_b, monkeypatch):
    rows, ab, _, kw = FORMS[name]
    ordinary = base._scales
    # base._case draws A's scales with seeds below 7400, B's from there
    monkeypatch.setattr(base, "_scales", lambda seed, shape, pow2: ordinary(seed, shape, pow2) * np.float32(2.0 ** (power_a if seed < 7400 else power_b)))
    got, z, _, st, _ = base._case(rows, 136, 400, ab, seed=9, **kw)
    assert st == tst.TST_OK
    # sums of 400 products of small integers whose scales lie within 2^12 of each other: whole multiples of the
    # least factor, fewer than 2^24 of them, hence exact in FP32
    assert np.abs(z).max() < 2.0 ** (power_a + power_b - 6 + 24) and np.isfinite(z).all() and np.array_equal(got, z), np.argwhere(got != z)[:5]
