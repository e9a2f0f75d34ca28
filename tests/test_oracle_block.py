"""Pins of oracle/block.py (CPU): the gradients of the norms, of the balance
loss and of the activations against central differences of the functions they
belong to, norms and activations against other ways to write them, and counts
against a walk over the tokens."""

import itertools

import numpy as np
import pytest

from oracle import block

H = 1e-5
# A central difference of a function with values and third derivatives of order 10
# is off by H^2 * 10 and 10 * 2^-52 / H.
CLOSE = 1e-7


def difference(f, v, at, h=H):
    up, down = v.copy(), v.copy()
    up[at] += h
    down[at] -= h
    return (f(up) - f(down)) / (2 * h)


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("gate", [None, "column", "token"])
def test_norm_gradients_against_differences(kind, post, gate):
    rng = np.random.default_rng(1)
    t, n = 3, 7
    v = {"y": rng.standard_normal((t, n)) + 0.3, "h": rng.standard_normal((t, n)), "weight": 1 + 0.3 * rng.standard_normal(n),
         "bias": rng.standard_normal(n)}
    if post:
        v["post_weight"] = 1 + 0.3 * rng.standard_normal(n)
    if gate:
        v["gate"] = rng.standard_normal(n if gate == "column" else (t, 1))
    opts = dict(post=post, kind=kind, eps=0.01, res_scale=0.7)
    dx, dr = rng.standard_normal((t, n)), rng.standard_normal((t, n))

    def total(**changed):
        r, x, _, _ = block.block_norm(**{**v, **changed}, **opts)
        return (dx * x).sum() + (dr * r).sum()

    r = block.block_norm(**v, **opts)[0]
    got = block.block_norm_bwd(dx, dr, r, v["y"], v["weight"], post_weight=v.get("post_weight"), gate=v.get("gate"), **opts)
    for name in v:
        grad = got["d" + name][0]
        assert grad.shape == v[name].shape
        for at in itertools.product(*map(range, v[name].shape)):
            assert abs(difference(lambda w: total(**{name: w}), v[name], at) - grad[at]) < CLOSE, (name, at)


def test_norms_have_unit_size():
    rng = np.random.default_rng(2)
    y = 3 * rng.standard_normal((5, 64)) + 2
    _, x, _, _ = block.block_norm(y, eps=1e-12)
    assert np.allclose((x ** 2).mean(1), 1.0)
    _, x, _, _ = block.block_norm(y, kind="layer", eps=1e-12)
    assert np.allclose(x.mean(1), 0.0) and np.allclose(x.var(1), 1.0)
    assert np.allclose(x, (y - y.mean(1, keepdims=True)) / y.std(1, keepdims=True))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_balance_gradient_against_differences(score):
    rng = np.random.default_rng(3)
    x, ids = rng.standard_normal((9, 5)), rng.integers(-1, 5, (9, 2))
    x[1, 2], x[4] = -np.inf, -np.inf
    offsets = [0, 4, 4, 8]
    counts, used, _ = block.balance(x, ids, offsets, score, 0.3)
    assert list(used) == [4, 0, 3]
    got, inside, _ = block.balance_bwd(x, counts, used, 2, offsets, score, 0.3, dloss=1.7)
    assert list(inside) == [True] * 8 + [False]
    for at in itertools.product(range(9), range(5)):
        if np.isneginf(x[at]):
            assert got[at] == 0
            continue
        # The counts do not move with the logits.
        d = difference(lambda v: 1.7 * block.balance(v, ids, offsets, score, 0.3)[2], x, at)
        assert abs(d - got[at]) < CLOSE


def test_balance_counts_and_even_load():
    rng = np.random.default_rng(4)
    x = rng.standard_normal((40, 6))
    ids = np.argsort(-x, 1)[:, :2]
    counts, used, loss = block.balance(x, ids)
    assert used[0] == 40 and all(counts[0][e] == sum(int(e in row) for row in ids) for e in range(6))
    even = np.arange(80).reshape(40, 2) % 6
    even[39] = [0, 3]  # 13 or 14 of each
    flat = block.balance(np.zeros((40, 6)), even)[2]
    assert abs(flat - 1.0) < 1e-12  # equal shares: sum_e f_e / experts = 1
    assert loss > 1.0  # choices follow the shares


def test_shares_of_small_scores():
    p = block.shares(np.array([[-800.0, -801.0, -np.inf], [5.0, -3.0, 0.0]]), "sigmoid")
    assert np.allclose(p[0], [1 / (1 + np.exp(-1)), 1 / (1 + np.exp(1)), 0])
    s = 1 / (1 + np.exp(-np.array([5.0, -3.0, 0.0])))
    assert np.allclose(p[1], s / s.sum())


@pytest.mark.parametrize("name", ["none", "relu", "silu", "gelu_tanh"])
def test_activations(name):
    z = np.concatenate([np.linspace(-9, 9, 181) + 0.013, [-40.0, 40.0]])
    want = {"none": z, "relu": np.where(z > 0, z, 0), "silu": z / (1 + np.exp(-z)),
            "gelu_tanh": 0.5 * z * (1 + np.tanh(np.sqrt(2 / np.pi) * (z + 0.044715 * z ** 3)))}[name]
    assert np.allclose(block.act(z, name), want, rtol=1e-12, atol=1e-14)
    for v, slope in zip(z, block.act_slope(z, name)):
        d = difference(lambda w: block.act(w, name)[0], np.array([v]), 0)
        assert abs(d - slope) < CLOSE
