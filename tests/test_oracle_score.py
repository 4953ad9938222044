"""The oracle of scored routing against brute force and differences (no GPU)."""
import itertools

import numpy as np
import pytest

from oracle import moe


@pytest.mark.parametrize("sigmoid", [True, False])
@pytest.mark.parametrize("groups,top_groups,best", [(1, 1, 1), (4, 2, 2), (4, 3, 1), (6, 1, 2)])
def test_choice_by_brute_force(sigmoid, groups, top_groups, best):
    rng = np.random.default_rng(groups + best)
    T, E, k = 40, 12, 2
    l, b = rng.normal(size=(T, E)), 0.05 * rng.normal(size=E)
    r = moe.route_scored(l, k, sigmoid, b, groups, top_groups, best, False, 1.5, 0.1)
    size = E // groups
    for t in range(T):
        s = 1 / (1 + np.exp(-l[t])) if sigmoid else np.exp(l[t]) / np.exp(l[t]).sum()
        c = s + b
        # the groups: the subset of the largest total value; then the subset of experts inside it
        value = [sum(sorted(c[g * size:(g + 1) * size])[-best:]) for g in range(groups)]
        keep = max(itertools.combinations(range(groups), top_groups), key=lambda gs: sum(value[g] for g in gs))
        inside = [e for e in range(E) if e // size in keep]
        pick = max(itertools.combinations(inside, k), key=lambda es: sum(c[e] for e in es))
        assert set(r["expert"][t]) == set(pick) and c[r["expert"][t][0]] >= c[r["expert"][t][1]]
        assert np.allclose(r["weight"][t], 1.5 * s[r["expert"][t]], rtol=1e-14)


@pytest.mark.parametrize("sigmoid", [True, False])
@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("shift", [0.0, -60.0])
def test_gradient_by_differences(sigmoid, normalize, shift):
    rng = np.random.default_rng(3)
    T, E, k = 6, 10, 3
    l = rng.normal(size=(T, E)) + shift
    l[2, 5] = -np.inf
    mask = np.array([1, 1, 1, 0, 1, 1])
    r = moe.route_scored(l, k, sigmoid, None, 2, 1, 2, normalize, 2.0, 0.3, mask)
    dw = rng.normal(size=(T, k))
    got, _ = moe.route_scored_backward(l, dw, 0.7, r, sigmoid, normalize, 2.0, 0.3, mask)
    f = lambda x: moe.route_scored_loss(x, dw, 0.7, r, sigmoid, normalize, 2.0, 0.3, mask)  # noqa: E731
    for t in range(T):
        for e in range(E):
            if l[t, e] == -np.inf:
                assert got[t, e] == 0.0
                continue
            h = 1e-5
            up, down = l.copy(), l.copy()
            up[t, e] += h
            down[t, e] -= h
            assert abs((f(up) - f(down)) / (2 * h) - got[t, e]) < 1e-8


def test_quantize_int8_values():
    q, s = moe.quantize_int8(np.array([[127.0, -63.5, 0.5, 0.0], [0.0, 0.0, 0.0, 0.0], [-1.0, 0.25, 1e-30, 0.5]]))
    assert q[0].tolist() == [127.0, -64.0, 0.0, 0.0] and s[0] == 1.0
    assert not q[1].any() and s[1] == np.float32(2.0 ** -96) / np.float32(127.0)
    assert q[2].tolist() == [-127.0, 32.0, 0.0, 64.0]   # 31.75 -> 32, 63.5 -> 64 (ties to even)
