"""The mixture-of-experts oracle against hand values, brute force and central differences."""
import numpy as np
import pytest

import synthetic
from oracle import moe


def _logits(seed, T, E):
    return synthetic.draw("normal", seed, T * E).reshape(T, E)


def test_route_hand_values():
    # token 0: a tie between experts 0 and 2 goes to 0 first; token 1 has one open expert; token 2
    # is closed by the mask; token 3 has no open expert
    ninf = -np.inf
    l = np.array([[1.0, 0.0, 1.0], [ninf, 2.0, ninf], [5.0, 5.0, 5.0], [ninf, ninf, ninf]])
    r = moe.route(l, 2, True, 0.5, mask=np.array([1, 1, 0, 1]))
    assert r["expert"].tolist() == [[0, 2], [1, -1], [-1, -1], [-1, -1]]
    assert r["counts"].tolist() == [1, 1, 1] and r["totals"].tolist() == [3, 2]
    assert r["row"].tolist() == [[0, 2], [1, -1], [-1, -1], [-1, -1]]
    assert np.allclose(r["weight"], [[0.5, 0.5], [1, 0], [0, 0], [0, 0]])
    # equal counts: the loss is coef * E * (1/3) * (sum of all probabilities) / n = 0.5 whatever p is
    assert abs(r["loss"] - 0.5) < 1e-15


def test_rows_are_a_permutation_by_expert_then_token():
    r = moe.route(_logits(1, 57, 9), 3, False, 0.1)
    flat = sorted((e, t) for t in range(57) for e in r["expert"][t])
    assert [int(r["row"][t, list(r["expert"][t]).index(e)]) for e, t in flat] == list(range(57 * 3))


@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("masked", [False, True])
def test_route_backward_against_differences(normalize, masked):
    T, E, k, coef = 6, 7, 3, 0.3
    l = _logits(2, T, E)
    l[1, 2] = -np.inf
    mask = np.array([1, 1, 0, 1, 1, 1]) if masked else None
    r = moe.route(l, k, normalize, coef, mask)
    dw = synthetic.draw("normal", 3, T * k).reshape(T, k)
    got, size = moe.route_backward(l, dw, 0.7, r, normalize, coef, mask)
    assert (np.abs(got) <= size + 1e-15).all()
    step = 1e-5
    for t in range(T):
        for e in range(E):
            if l[t, e] == -np.inf:
                assert got[t, e] == 0
                continue
            hi, lo = l.copy(), l.copy()
            hi[t, e] += step
            lo[t, e] -= step
            want = (moe.route_loss(hi, dw, 0.7, r, normalize, coef, mask) -
                    moe.route_loss(lo, dw, 0.7, r, normalize, coef, mask)) / (2 * step)
            assert abs(got[t, e] - want) < 1e-9, (t, e)


def test_round_e4m3_lists_every_code():
    # every positive finite e4m3 value by its definition; the midpoints go to the even mantissa
    vals = sorted({(m / 8.0) * 2.0 ** -6 for m in range(8)} |
                  {(1 + m / 8.0) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)} - {480.0})
    assert len(vals) == 127 and vals[-1] == 448.0
    assert np.array_equal(moe.round_e4m3(vals), vals)
    mid = (np.array(vals[:-1]) + np.array(vals[1:])) / 2
    got = moe.round_e4m3(mid)
    even = [vals[i] if i % 2 == 0 else vals[i + 1] for i in range(len(mid))]
    assert np.array_equal(got, even)
    assert np.array_equal(moe.round_e4m3([1e9, -500.0, 0.0]), [448.0, -448.0, 0.0])


def test_quantize_reproduces_within_half_a_step():
    x = synthetic.draw("normal", 4, 5 * 300).reshape(5, 300).astype(np.float32)
    x[2, 128:256] = 0
    q, s = moe.quantize(x)
    assert s.shape == (5, 3)
    back = q * np.repeat(s.astype(np.float64), 128, axis=1)[:, :300]
    # half of e4m3's relative step (2^-4), or half its least step (2^-10 of the scale)
    assert (np.abs(back - x) <= 2.0 ** -4 * np.abs(x) * (1 + 1e-6) +
            2.0 ** -10 * np.repeat(s.astype(np.float64), 128, axis=1)[:, :300]).all()
    assert (back[2, 128:256] == 0).all()


def test_combine_and_its_gradient():
    r = moe.route(_logits(5, 11, 4), 2, True, 0.0)
    rows = synthetic.draw("normal", 6, 22 * 5).reshape(22, 5)
    out, size = moe.combine(rows, r["row"], r["weight"])
    want = np.array([sum(r["weight"][t, j] * rows[r["row"][t, j]] for j in range(2)) for t in range(11)])
    assert np.allclose(out, want) and (np.abs(out) <= size + 1e-15).all()
    d = synthetic.draw("normal", 7, 55).reshape(11, 5)
    d_rows, d_w, _ = moe.combine_backward(rows, r["row"], r["weight"], d)
    step = 1e-6
    for i in (0, 9, 21):
        for h in range(5):
            hi, lo = rows.copy(), rows.copy()
            hi[i, h] += step
            lo[i, h] -= step
            diff = np.sum(d * (moe.combine(hi, r["row"], r["weight"])[0] - moe.combine(lo, r["row"], r["weight"])[0]))
            assert abs(d_rows[i, h] - diff / (2 * step)) < 1e-8
    for t in (0, 10):
        for j in range(2):
            hi, lo = r["weight"].copy(), r["weight"].copy()
            hi[t, j] += step
            lo[t, j] -= step
            diff = np.sum(d * (moe.combine(rows, r["row"], hi)[0] - moe.combine(rows, r["row"], lo)[0]))
            assert abs(d_w[t, j] - diff / (2 * step)) < 1e-8
