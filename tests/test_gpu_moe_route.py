"""GPU expert routing (dg_moe_route*, dg_moe_route_bwd*) against oracle/moe.py.

Ids must equal the oracle's wherever its choice does not hang on differences
of 1e-5 between scores; weights are held to 2^-18 of their value (float32
exponents of up to 32 magnitude carry 2^-19, sums and quotients a few 2^-23);
gradients to 2^-15 of the largest term that enters them.
"""

import numpy as np
import pytest
import torch

from oracle import moe
from tests.gpu_util import require_gpu

pytestmark = pytest.mark.gpu


def _strided(x, pad):
    out = torch.full((x.shape[0], x.shape[1] + pad), 77.0, dtype=x.dtype, device="cuda")
    out[:, :x.shape[1]] = x
    return out[:, :x.shape[1]]


def _run(dg, x, topk, bf16=False, pad=0, **kw):
    t = torch.as_tensor(x, dtype=torch.bfloat16 if bf16 else torch.float32, device="cuda")
    t = _strided(t, pad) if pad else t
    ids = torch.full((x.shape[0], topk), -7, dtype=torch.int32, device="cuda")
    w = torch.full((x.shape[0], topk), float("nan"), device="cuda")
    bias = kw.pop("bias", None)
    bias = None if bias is None else torch.as_tensor(bias, dtype=torch.float32, device="cuda")
    (dg.dg_moe_route_bf16 if bf16 else dg.dg_moe_route)(t, ids, w, bias=bias, **kw)
    return ids.cpu().numpy(), w.cpu().numpy().astype(np.float64)


def _bf(x):
    return torch.as_tensor(x, dtype=torch.float32).bfloat16().float().numpy()


def _oracle_args(kw):
    return dict(score=kw.get("score", "softmax"), groups=kw.get("expert_groups", 1), topk_groups=kw.get("topk_groups", 1),
                group_top=kw.get("group_top", 2))


def _check(dg, x, topk, bf16, pad, kw, gap=1e-5):
    bias = kw.get("bias")
    ids, w = _run(dg, x, topk, bf16, pad, **kw)
    ref_ids, ref_w = moe.route(x, topk, bias=bias, renormalize=kw.get("renormalize", True), scale=kw.get("scale", 1.0),
                               **_oracle_args(kw))
    fine = moe.settled(x, topk, bias=bias, gap=gap, **_oracle_args(kw))
    assert fine.mean() > 0.9
    assert np.array_equal(ids[fine], ref_ids[fine])
    assert np.all(np.abs(w[fine] - ref_w[fine]) <= 2.0 ** -18 * np.abs(ref_w[fine]) + 1e-30)
    assert np.array_equal(w == 0, (ids < 0) | (w == 0)) and np.all(w[ids < 0] == 0)
    return ids


CASES = [  # experts, topk, tokens, options
    (1, 1, 3, {}),
    (2, 2, 1, dict(score="sigmoid", renormalize=False)),
    (5, 3, 130, dict(scale=2.5)),
    (64, 8, 33, dict(score="sigmoid", bias=True)),
    (65, 32, 9, {}),
    (72, 6, 257, dict(renormalize=False)),
    (160, 6, 64, dict(expert_groups=8, topk_groups=3, group_top=1)),
    (256, 8, 129, dict(score="sigmoid", bias=True, expert_groups=8, topk_groups=4, scale=2.5)),
    (256, 8, 64, dict(bias=True, expert_groups=64, topk_groups=5)),
    (255, 10, 31, dict(score="sigmoid", bias=True, expert_groups=3, topk_groups=2, group_top=1)),
    (257, 4, 17, dict(score="sigmoid", bias=True)),
    (512, 8, 20, dict(score="sigmoid", bias=True, expert_groups=8, topk_groups=8)),
    (1000, 7, 11, dict(expert_groups=20, topk_groups=4)),
    (1024, 32, 6, dict(bias=True)),
    (12, 12, 40, dict(expert_groups=12, topk_groups=5, score="sigmoid", bias=True)),
]


@pytest.mark.parametrize("bf16,pad", [(False, 0), (False, 3), (True, 0), (True, 5)])
@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{c[0]}x{c[1]}x{c[2]}")
def test_route(case, bf16, pad):
    dg = require_gpu()
    experts, topk, tokens, kw = case
    rng = np.random.default_rng(experts * 31 + topk)
    x = _bf(1.5 * rng.standard_normal((tokens, experts)))
    kw = dict(kw)
    if kw.get("bias"):
        kw["bias"] = (0.2 * rng.standard_normal(experts)).astype(np.float32)
    _check(dg, x, topk, bf16, pad, kw, gap=1e-6)


@pytest.mark.parametrize("kw", [
    {}, dict(score="sigmoid"), dict(score="sigmoid", bias=True, expert_groups=8, topk_groups=3),
    dict(expert_groups=8, topk_groups=2, group_top=1)], ids=str)
def test_masked_experts_and_rows(kw):
    dg = require_gpu()
    rng = np.random.default_rng(8)
    x = _bf(rng.standard_normal((96, 64)))
    x[rng.random(x.shape) < 0.7] = -np.inf       # often fewer than topk experts left
    x[::5] = -np.inf                             # nothing left
    x[1::10, 1:] = -np.inf                       # one expert left
    x[1::10, 0] = -3.0e38                        # and that of the type's lowest order, yet not masked
    kw = dict(kw)
    if kw.get("bias"):
        kw["bias"] = (0.2 * rng.standard_normal(64)).astype(np.float32)
    ids = _check(dg, x, 8, False, 0, kw)
    assert np.all(ids[::5] == -1)
    assert np.all(ids[1::10, 0] == 0) and np.all(ids[1::10, 1:] == -1)


def test_ties_go_to_the_lowest_index():
    dg = require_gpu()
    rng = np.random.default_rng(9)
    x = rng.integers(-2, 3, (64, 200)).astype(np.float32)
    x[x == 0] *= rng.choice([-1.0, 1.0], int((x == 0).sum()))  # +0 and -0 are equal
    for kw in ({}, dict(score="sigmoid", bias=np.zeros(200, dtype=np.float32)),
               dict(score="sigmoid", expert_groups=10, topk_groups=3)):
        ids, _ = _run(dg, x, 16, **kw)
        ref, _ = moe.route(x, 16, bias=kw.get("bias"), **_oracle_args(kw))
        assert np.array_equal(ids, ref)


def test_extreme_logits():
    dg = require_gpu()
    x = np.array([[1e4, -1e4, 0, 5, 3e38, -3e38, 1, 2], [np.inf, 0, 1, 2, 3, 4, 5, 6], [-1e4] * 8, [88, 89, 90, 91, 92, 93, 94, 95]],
                 dtype=np.float32)
    for score in ("softmax", "sigmoid"):
        ids, w = _run(dg, x, 4, score=score)
        ref, ref_w = moe.route(x, 4, score)
        assert np.array_equal(ids, ref)
        fine = np.isfinite(ref_w).all(1)
        if score == "softmax":
            assert not fine[1] and np.isnan(w[1]).all()
        # exp(-1e4) underflows in float32: those sigmoids are 0 and so are their weights
        fine[2] &= score == "softmax"
        assert np.all(np.abs(w[fine] - ref_w[fine]) <= 2.0 ** -18 * ref_w[fine] + 1e-37)
        if score == "sigmoid":
            assert np.all(w[2] == 0)


def test_nan_logits_choose_valid_experts():
    dg = require_gpu()
    rng = np.random.default_rng(10)
    x = rng.standard_normal((64, 100)).astype(np.float32)
    x[rng.random(x.shape) < 0.3] = np.nan
    x[0] = np.nan
    for kw in ({}, dict(score="sigmoid"), dict(score="sigmoid", bias=np.zeros(100, dtype=np.float32), expert_groups=10, topk_groups=4)):
        ids, _ = _run(dg, x, 8, **kw)
        assert np.all(ids[0] == -1)
        for t in range(1, 64):
            live = ids[t][ids[t] >= 0]
            assert len(set(live)) == len(live) and np.all(live < 100) and not np.isnan(x[t, live]).any()
    _, w = _run(dg, x, 8)
    assert np.isnan(w[1:]).all()


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [False, True])
@pytest.mark.parametrize("experts,topk,tokens", [(1, 1, 2), (7, 7, 5), (64, 8, 130), (72, 6, 33), (256, 8, 65), (1000, 32, 9)])
def test_route_bwd(bf16, score, renormalize, experts, topk, tokens):
    dg = require_gpu()
    rng = np.random.default_rng(experts + topk)
    x = _bf(1.5 * rng.standard_normal((tokens, experts)))
    if experts > 40:
        x[rng.random(x.shape) < 0.1] = -np.inf
    ids, _ = moe.route(x, topk, score)
    ids[0, -1] = -1
    ids[-1, 0] = experts + 5  # names no expert
    dw = rng.standard_normal((tokens, topk)).astype(np.float32)
    dt = torch.bfloat16 if bf16 else torch.float32
    logits = _strided(torch.as_tensor(x, device="cuda").to(dt), 3)
    dx = _strided(torch.full((tokens, experts), float("nan"), dtype=dt, device="cuda"), 1)
    (dg.dg_moe_route_bwd_bf16 if bf16 else dg.dg_moe_route_bwd)(
        logits, torch.as_tensor(ids, dtype=torch.int32, device="cuda"), torch.as_tensor(dw, device="cuda"), dx, score=score,
        renormalize=renormalize, scale=2.5)
    got = dx.float().cpu().numpy().astype(np.float64)
    ref = moe.route_bwd(x, ids, dw, score, renormalize, 2.5)
    s = moe.scores(x, score)
    chosen = np.where((ids >= 0) & (ids < experts), np.take_along_axis(s, np.clip(ids, 0, experts - 1), 1), 0.0).sum(1, keepdims=True)
    div = np.where(chosen > 0, chosen, 1.0) if renormalize else 1.0
    bound = 2.0 ** -15 * 2.5 * np.abs(dw).max(1, keepdims=True) / div * s + 1e-30
    if bf16:
        bound = bound + 2.0 ** -8 * np.abs(ref)
    assert np.all(np.abs(got - ref) <= bound)


def test_route_bwd_against_differences():
    """The gradient against central differences of dg_moe_route's own weights:
    steps of 2^-6 leave h^2/6 third derivatives (below 1e-4 here) and float32
    noise of 2^-22 / 2^-6 a difference."""
    dg = require_gpu()
    rng = np.random.default_rng(12)
    tokens, experts, topk, h = 8, 16, 4, 2.0 ** -6
    x = np.stack([rng.permutation(experts) * 0.25 for _ in range(tokens)]).astype(np.float32)  # steps never reorder
    dw = rng.standard_normal((tokens, topk)).astype(np.float32)
    for score in ("softmax", "sigmoid"):
        ids, _ = _run(dg, x, topk, score=score)
        dx = torch.empty(tokens, experts, device="cuda")
        dg.dg_moe_route_bwd(torch.as_tensor(x, device="cuda"), torch.as_tensor(ids, device="cuda"),
                            torch.as_tensor(dw, device="cuda"), dx, score=score)
        got = dx.cpu().numpy()
        for e in range(experts):
            f = []
            for sign in (1, -1):
                y = x.copy()
                y[:, e] += sign * h
                i2, w = _run(dg, y, topk, score=score)
                assert np.array_equal(i2, ids)
                f.append((w * dw).sum(1))
            assert np.all(np.abs((f[0] - f[1]) / (2 * h) - got[:, e]) < 5e-4)


def test_many_tokens_and_no_tokens():
    dg = require_gpu()
    x = torch.randn(70000, 32, device="cuda")
    ids = torch.empty(70000, 2, dtype=torch.int32, device="cuda")
    w = torch.empty(70000, 2, device="cuda")
    dg.dg_moe_route(x, ids, w)
    ref = x.sort(dim=1, descending=True, stable=True).indices[:, :2]
    assert torch.equal(ids.long(), ref)
    dg.dg_moe_route(x[:0], ids[:0], w[:0])


@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("experts,groups,keep", [(34, 2, 1), (92, 4, 2), (184, 8, 3), (192, 6, 2), (500, 4, 2), (1016, 8, 4),
                                                 (96, 32, 7), (62, 31, 9), (1024, 64, 11)])
def test_groups_of_any_size(experts, groups, keep, bias):
    """Groups that fill their lanes and groups that do not, few and many, some with every expert masked."""
    dg = require_gpu()
    rng = np.random.default_rng(experts + groups)
    x = _bf(1.5 * rng.standard_normal((67, experts)))
    x[:20, :experts // groups] = -np.inf
    x[20:40][rng.random((20, experts)) < 0.5] = -np.inf
    kw = dict(score="sigmoid", expert_groups=groups, topk_groups=keep, scale=2.5)
    if bias:
        kw["bias"] = (0.2 * rng.standard_normal(experts)).astype(np.float32)
    for group_top in (1, 2):
        _check(dg, x, min(8, keep * (experts // groups)), False, 0, dict(kw, group_top=group_top), gap=1e-6)
