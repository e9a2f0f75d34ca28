"""GPU routing gradient (dg_moe_route_bwd*) where float32 has little room:
chosen scores whose sum is tiny.

Bounds.  A score carries 2^-18 of its value (float32 exponents of up to 104 in
magnitude carry 2^-19, the sum, the quotient and the reciprocal a few 2^-23)
and, below the normal range, 2^-149; a weight r = s / S of k chosen experts
therefore 2^-17 of its value and (k + 1) 2^-149 / S, and both enter the gradient
r (dw - sum dw r) twice.
"""

import numpy as np
import pytest
import torch

from oracle import moe
from tests.gpu_util import require_gpu

pytestmark = pytest.mark.gpu


def _bwd(dg, x, ids, dw, bf16=False, **kw):
    dt = torch.bfloat16 if bf16 else torch.float32
    logits = torch.as_tensor(x, device="cuda").to(dt)
    dx = torch.full_like(logits, float("nan"))
    (dg.dg_moe_route_bwd_bf16 if bf16 else dg.dg_moe_route_bwd)(
        logits, torch.as_tensor(ids, dtype=torch.int32, device="cuda"), torch.as_tensor(dw, device="cuda"), dx, **kw)
    return dx.float().cpu().numpy().astype(np.float64)


def _weight_bound(x, ids, dw, score, scale):
    """Error of scale * r (dw - sum dw r) at the chosen experts, scattered over the row."""
    s = np.take_along_axis(moe.scores(x, score), ids, 1)
    total = s.sum(1, keepdims=True)
    most = np.abs(dw).max(1, keepdims=True)
    part = 4 * scale * most * (2.0 ** -17 * s / total + (ids.shape[1] + 1) ** 2 * 2.0 ** -149 / total) + 1e-30
    full = np.zeros(x.shape)
    np.put_along_axis(full, ids, part, 1)
    return full


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("experts,topk", [(4, 4), (64, 8), (72, 6), (256, 8), (1000, 32)])
@pytest.mark.parametrize("low,high", [(-91.0, -88.0), (-97.0, -88.0), (-60.0, -50.0)])
def test_tiny_sigmoids(low, high, experts, topk, bf16):
    """All experts far below zero: the chosen sigmoids' sum is near or below the
    smallest normal number, the renormalised weights and their gradient are not."""
    dg = require_gpu()
    rng = np.random.default_rng(experts + topk)
    x = rng.uniform(low, high, (33, experts)).astype(np.float32)
    x = torch.as_tensor(x).bfloat16().float().numpy() if bf16 else x
    ids, _ = moe.route(x, topk, "sigmoid")
    dw = rng.standard_normal(ids.shape).astype(np.float32)
    got = _bwd(dg, x, ids, dw, bf16, score="sigmoid", scale=2.5)
    ref = moe.route_bwd(x, ids, dw, "sigmoid", True, 2.5)
    assert np.all(np.abs(got - ref) <= _weight_bound(x, ids, dw, "sigmoid", 2.5) + (2.0 ** -8 * np.abs(ref) if bf16 else 0))


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("experts,topk", [(5, 3), (64, 8), (72, 6), (256, 8), (1000, 32)])
@pytest.mark.parametrize("below", [5.0, 60.0, 92.0])
def test_softmax_of_tiny_chosen_scores(below, experts, topk, bf16):
    """One expert far above the chosen ones, as a selection bias makes it: the
    gradient stays with the chosen experts and is exactly zero at the others."""
    dg = require_gpu()
    rng = np.random.default_rng(experts * 3 + topk)
    x = rng.uniform(-2.0, 2.0, (33, experts)).astype(np.float32) - np.float32(below)
    x[:, 1] = 0.0
    x = torch.as_tensor(x).bfloat16().float().numpy() if bf16 else x
    ids = np.stack([rng.permutation(np.delete(np.arange(experts), 1))[:topk] for _ in range(len(x))])
    dw = rng.standard_normal(ids.shape).astype(np.float32)
    got = _bwd(dg, x, ids, dw, bf16, score="softmax", scale=2.5)
    ref = moe.route_bwd(x, ids, dw, "softmax", True, 2.5)
    chosen = np.zeros(x.shape, dtype=bool)
    np.put_along_axis(chosen, ids, True, 1)
    assert np.all(got[~chosen] == 0)
    bound = _weight_bound(x, ids, dw, "softmax", 2.5) + (2.0 ** -8 * np.abs(ref) if bf16 else 0)
    assert np.all(np.abs(got - ref)[chosen] <= bound[chosen])


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_scores_that_underflow_have_no_gradient(score):
    dg = require_gpu()
    x = np.full((3, 64), -2000.0, dtype=np.float32)
    x[:, 9] = 0.0
    ids = np.array([[3, 4], [5, -1], [63, 0]])
    got = _bwd(dg, x, ids, np.ones((3, 2), dtype=np.float32), score=score)
    assert np.all(got == 0)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("renormalize", [False, True])
@pytest.mark.parametrize("experts,topk", [(1, 1), (5, 3), (64, 8), (72, 6), (256, 8), (1000, 32)])
def test_slope_of_saturated_sigmoids(experts, topk, renormalize, bf16):
    """Logits up to 40 of both signs: s (1 - s) keeps its relative accuracy where
    1 - s is far below one unit in the last place of s.  Exponents of up to 58 in
    magnitude carry 2^-19, the rest a few 2^-23."""
    dg = require_gpu()
    rng = np.random.default_rng(experts * 7 + topk)
    x = rng.uniform(-40.0, 40.0, (65, experts)).astype(np.float32)
    x[::3] = np.abs(x[::3])
    x = torch.as_tensor(x).bfloat16().float().numpy() if bf16 else x
    ids = np.stack([rng.permutation(experts)[:topk] for _ in range(len(x))])
    dw = rng.standard_normal(ids.shape).astype(np.float32)
    got = np.take_along_axis(_bwd(dg, x, ids, dw, bf16, score="sigmoid", renormalize=renormalize, scale=2.5), ids, 1)
    ref = np.take_along_axis(moe.route_bwd(x, ids, dw, "sigmoid", False, 1.0), ids, 1)  # dw s (1 - s)
    s = np.take_along_axis(moe.scores(x, "sigmoid"), ids, 1)
    rest = np.take_along_axis(moe.scores(-x, "sigmoid"), ids, 1)
    if renormalize:
        r = s / s.sum(1, keepdims=True)
        ref = 2.5 * r * (dw - (dw * r).sum(1, keepdims=True)) * rest
        bound = 2.0 ** -17 * 2.5 * r * rest * (np.abs(dw) + (np.abs(dw) * r).sum(1, keepdims=True))
    else:
        ref = 2.5 * dw * s * rest
        bound = 2.0 ** -18 * np.abs(ref)
    assert np.all(np.abs(got - ref) <= bound + (2.0 ** -8 * np.abs(ref) if bf16 else 0) + 1e-37)


def test_slope_past_the_range_of_the_exponent():
    """Logits of 60 to 3e38: 1 - s goes down to float32's smallest numbers and to 0, never below."""
    dg = require_gpu()
    x = np.array([[60.0, 80.0, 85.0, 88.0, 95.0, 200.0, 3e38, np.inf], [-60.0, -80.0, -85.0, -88.0, -95.0, -200.0, -3e38, -np.inf]],
                 dtype=np.float32)
    ids = np.tile(np.arange(8), (2, 1))
    got = _bwd(dg, x, ids, np.ones((2, 8), dtype=np.float32), score="sigmoid", renormalize=False)
    e = np.exp(-np.abs(x.astype(np.float64)))
    ref = e / (1.0 + e) ** 2
    assert np.all(got >= 0) and np.all(np.abs(got - ref) <= 2.0 ** -17 * ref + 2.0 ** -147)


@pytest.mark.parametrize("renormalize", [False, True])
def test_nan_logit_of_a_given_expert_shows(renormalize):
    """ids that name an expert whose logit is NaN: its own score is NaN, and with it
    all of the token's renormalised weights; other tokens keep their gradient."""
    dg = require_gpu()
    rng = np.random.default_rng(3)
    x = rng.standard_normal((3, 16)).astype(np.float32)
    x[1, 5] = np.nan
    ids = np.array([[5, 2, 9]] * 3)
    got = _bwd(dg, x, ids, np.tile(np.float32([1, 2, 3]), (3, 1)), score="sigmoid", renormalize=renormalize)
    want = np.zeros((3, 16), dtype=bool)
    want[1, [5, 2, 9] if renormalize else [5]] = True
    assert np.array_equal(np.isnan(got), want)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [False, True])
@pytest.mark.parametrize("experts,topk,tokens", [(64, 8, 130), (72, 6, 33), (128, 2, 9), (256, 8, 65), (504, 4, 7), (1000, 32, 9), (1024, 8, 5)])
def test_rows_without_gaps(bf16, score, renormalize, experts, topk, tokens):
    """Whole vectors of a row's logits: the bits of rows with gaps, and the formula's
    values to 2^-15 of the largest term."""
    dg = require_gpu()
    rng = np.random.default_rng(experts + 5 * topk)
    x = torch.as_tensor(1.5 * rng.standard_normal((tokens, experts)), dtype=torch.float32).bfloat16().float().numpy()
    x[rng.random(x.shape) < 0.1] = -np.inf
    ids, _ = moe.route(x, topk, score)
    ids[0, -1] = -1
    ids[-1, 0] = experts + 5  # names no expert
    dw = rng.standard_normal((tokens, topk)).astype(np.float32)
    got = _bwd(dg, x, ids, dw, bf16, score=score, renormalize=renormalize, scale=2.5)
    dt = torch.bfloat16 if bf16 else torch.float32
    wide, gap = (torch.full((tokens, experts + n), float("nan"), dtype=dt, device="cuda") for n in (3, 1))
    wide[:, :experts] = torch.as_tensor(x, device="cuda")
    (dg.dg_moe_route_bwd_bf16 if bf16 else dg.dg_moe_route_bwd)(
        wide[:, :experts], torch.as_tensor(ids, dtype=torch.int32, device="cuda"), torch.as_tensor(dw, device="cuda"),
        gap[:, :experts], score=score, renormalize=renormalize, scale=2.5)
    assert np.array_equal(gap[:, :experts].float().cpu().numpy().astype(np.float64), got) and bool(gap[:, experts:].isnan().all())
    ref = moe.route_bwd(x, ids, dw, score, renormalize, 2.5)
    s = moe.scores(x, score)
    chosen = np.where((ids >= 0) & (ids < experts), np.take_along_axis(s, np.clip(ids, 0, experts - 1), 1), 0.0).sum(1, keepdims=True)
    div = np.where(chosen > 0, chosen, 1.0) if renormalize else 1.0
    bound = 2.0 ** -15 * 2.5 * np.abs(dw).max(1, keepdims=True) / div * s + 1e-30 + (2.0 ** -8 * np.abs(ref) if bf16 else 0)
    assert np.all(np.abs(got - ref) <= bound)


@pytest.mark.parametrize("experts,topk", [(4, 4), (72, 6), (256, 8)])
@pytest.mark.parametrize("low,high", [(-97.0, -88.0), (-87.0, -60.0)])
def test_weights_of_tiny_sigmoids(low, high, experts, topk):
    """The weights whose gradient test_tiny_sigmoids takes, to the same accuracy."""
    dg = require_gpu()
    rng = np.random.default_rng(experts + topk)
    x = rng.uniform(low, high, (33, experts)).astype(np.float32)
    ref_ids, ref = moe.route(x, topk, "sigmoid", scale=2.5)
    ids, w = torch.empty(33, topk, dtype=torch.int32, device="cuda"), torch.empty(33, topk, device="cuda")
    dg.dg_moe_route(torch.as_tensor(x, device="cuda"), ids, w, score="sigmoid", scale=2.5)
    assert np.array_equal(ids.cpu().numpy(), ref_ids)
    total = np.take_along_axis(moe.scores(x, "sigmoid"), ref_ids, 1).sum(1, keepdims=True)
    assert np.all(np.abs(w.cpu().numpy() - ref) <= 2.0 ** -17 * ref + 2.5 * (topk + 1) * 2.0 ** -149 / total)
