"""Pins of oracle/moe.py (CPU): gradients against central differences of the
functions they belong to, the routing choice against a search over all
subsets, the row plan against its own inverse and the layout's rules."""

import itertools

import numpy as np
import pytest

from oracle import moe


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [False, True])
def test_route_gradient_against_differences(score, renormalize):
    rng = np.random.default_rng(3)
    x, dw = rng.standard_normal((4, 9)), rng.standard_normal((4, 3))
    ids, _ = moe.route(x, 3, score)
    ids[2, 1] = -1
    got = moe.route_bwd(x, ids, dw, score, renormalize, 2.5)
    h = 1e-6
    for t, e in itertools.product(range(4), range(9)):
        up, down = x.copy(), x.copy()
        up[t, e] += h
        down[t, e] -= h
        f = [(moe.weights_of(v, ids, score, renormalize, 2.5) * dw).sum() for v in (up, down)]
        # central difference: O(h^2) truncation and 1e-16 / h rounding
        assert abs((f[0] - f[1]) / (2 * h) - got[t, e]) < 1e-8


def test_route_choice_against_all_subsets():
    rng = np.random.default_rng(4)
    for trial in range(40):
        x, bias = rng.standard_normal((1, 8)), 0.3 * rng.standard_normal(8)
        ids, w = moe.route(x, 3, "sigmoid", bias, groups=4, topk_groups=2, group_top=2)
        key = moe.scores(x, "sigmoid")[0] + bias
        pairs = key.reshape(4, 2).sum(1)
        groups = max(itertools.combinations(range(4), 2), key=lambda c: sum(pairs[list(c)]))
        allowed = [e for e in range(8) if e // 2 in groups]
        best = max(itertools.combinations(allowed, 3), key=lambda c: sum(key[list(c)]))
        assert set(ids[0]) == set(best)
        assert np.all(np.diff(key[ids[0]]) < 0)
        assert abs(w.sum() - 1) < 1e-12


def test_route_ties_and_masks():
    x = np.zeros((3, 6))
    x[1, :3] = -np.inf
    x[2] = -np.inf
    ids, w = moe.route(x, 4, "softmax")
    assert ids[0].tolist() == [0, 1, 2, 3] and ids[1].tolist() == [3, 4, 5, -1] and ids[2].tolist() == [-1] * 4
    assert w[1, 3] == 0 and np.all(w[2] == 0) and np.allclose(w[0], 0.25)


def test_plans_are_inverse_and_aligned():
    rng = np.random.default_rng(5)
    ids = rng.integers(-1, 9, (300, 3)).astype(np.int32)
    rows, src, m_indices, off = moe.plan_contiguous(ids, 2, 5, 1280)
    used = np.flatnonzero(src >= 0)
    assert np.array_equal(rows.reshape(-1)[src[used]], used)
    assert np.array_equal(ids.reshape(-1)[src[used]] - 2, m_indices[used])
    assert np.all(off % 128 == 0) and np.array_equal((rows >= 0), (ids >= 2) & (ids < 7))
    for g in range(5):
        assert np.all(np.diff(src[(m_indices == g)]) > 0)
    rows, src, count = moe.plan_masked(ids, 2, 5, 32)
    assert np.all(count <= 32) and np.array_equal(np.bincount(np.flatnonzero(src >= 0) // 32, minlength=5), count)


def test_swiglu_gradient_against_differences():
    rng = np.random.default_rng(6)
    h, da = rng.standard_normal((3, 8)) * 2, rng.standard_normal((3, 4))
    got = moe.swiglu_bwd(h, da)
    for i, j in itertools.product(range(3), range(8)):
        up, down = h.copy(), h.copy()
        up[i, j] += 1e-6
        down[i, j] -= 1e-6
        assert abs(((moe.swiglu(up) - moe.swiglu(down)) * da).sum() / 2e-6 - got[i, j]) < 1e-8


def test_combine_gradient_against_differences():
    rng = np.random.default_rng(7)
    d, w, dy = rng.standard_normal((6, 4)), rng.random((3, 2)), rng.standard_normal((3, 4))
    rows = np.array([[0, 5], [3, -1], [1, 2]])
    src = np.full(6, -1)
    for i, r in enumerate(rows.reshape(-1)):
        if r >= 0:
            src[r] = i
    dd, dw, _ = moe.combine_bwd(dy, d, src, rows, w)
    f = lambda d, w: (moe.combine(d, rows, w)[0] * dy).sum()  # noqa: E731
    h = 1e-6
    for r, c in itertools.product(range(6), range(4)):
        a, b = d.copy(), d.copy()
        a[r, c] += h
        b[r, c] -= h
        assert abs((f(a, w) - f(b, w)) / (2 * h) - dd[r, c]) < 1e-8
    for t, j in itertools.product(range(3), range(2)):
        a, b = w.copy(), w.copy()
        a[t, j] += h
        b[t, j] -= h
        assert abs((f(d, a) - f(d, b)) / (2 * h) - dw[t, j]) < 1e-8


def test_half_step():
    from oracle import e4m3
    grid = np.unique(np.abs(e4m3.decode(np.arange(127, dtype=np.uint8)).astype(np.float64)))
    mids = (grid[1:] + grid[:-1]) / 2
    assert np.array_equal(moe.half_step(mids), (grid[1:] - grid[:-1]) / 2)
