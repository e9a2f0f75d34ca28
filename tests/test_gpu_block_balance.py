"""GPU load balance of a router (dg_moe_balance*, dg_moe_balance_bwd*) against
oracle/block.py.

Counts and tokens in use are whole numbers and must be equal.  Shares are float32:
an exponential is within 2 ulp and 2^-24 of the distance to the largest logit (at
most 2^5 here for scores that matter), sums of up to 1024 of them are 16 values a
lane and 6 steps between lanes, so a share loses at most 2^-17 of itself; the loss
adds chunks of 8 tokens a wave and up to 16 + 64 rows, all positive: 2^-16 of it.
The gradient is share times (f - mean f): 2^-16 of the share times (f + mean f),
then the added gradient and, for bf16, one rounding.
"""

import numpy as np
import pytest
import torch

from oracle import block
from tests.block_util import workspace
from tests.gpu_util import bf16_to_f64, dev, host, require_gpu

pytestmark = pytest.mark.gpu

LOST = 2.0 ** -16


def make(rng, tokens, experts, topk, bf16, masked=0.1):
    x = (2 * rng.standard_normal((tokens, experts))).astype(np.float32)
    if masked and tokens > 3:
        x[rng.random(x.shape) < masked] = -np.inf
        x[rng.random(tokens) < masked] = -np.inf
    ids = np.array([rng.permutation(experts)[:topk] for _ in range(tokens)], dtype=np.int32).reshape(tokens, topk)
    ids[rng.random(ids.shape) < 0.1] = -1
    if tokens > 1:
        ids[1, 0] = 2 ** 31 - 1  # names no expert
    bits = (x.view(np.uint32) >> 16).astype(np.uint16) if bf16 else x
    return bits, (bf16_to_f64(bits) if bf16 else x.astype(np.float64)), ids


def on_device(v, ld):
    """The matrix with rows ld apart, NaN between them."""
    pad = np.full((v.shape[0], ld), 0x7FC0, dtype=np.uint16) if v.dtype == np.uint16 else np.full((v.shape[0], ld), np.nan, dtype=np.float32)
    pad[:, :v.shape[1]] = v
    t = dev(pad)
    return (t.view(torch.bfloat16) if v.dtype == np.uint16 else t)[:, :v.shape[1]]


def cuts(rng, tokens, seqs):
    """Offsets of sequences with empty ones, from behind the first token to before the last."""
    if not seqs:
        return None
    lo, hi = min(2, tokens), max(min(2, tokens), tokens - 3)
    inner = np.sort(rng.integers(lo, hi + 1, seqs - 1))
    off = np.concatenate([[lo], inner, [hi]]).astype(np.int32)
    if seqs > 3:
        off[2] = off[1]
    return off


def close(got, want, mag, what, extra=0.0):
    bad = ~(np.abs(got - want) <= LOST * mag + extra + 2.0 ** -149)
    assert not bad.any(), f"{what}: {bad.sum()}, first at {np.argwhere(bad)[0]}"


SIZES = [(0, 8, 2, 0, 8), (1, 1, 1, 0, 1), (1, 256, 8, 0, 256), (2, 3, 3, 1, 5), (33, 64, 4, 0, 64), (70, 72, 6, 5, 73), (300, 128, 8, 9, 132),
         (513, 500, 32, 0, 501), (1000, 256, 8, 700, 256), (2000, 16, 2, 3, 16), (700, 1024, 8, 4, 1024), (4099, 60, 5, 1, 60)]


@pytest.mark.parametrize("tokens,experts,topk,seqs,ld", SIZES, ids=str)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bf16", [False, True])
def test_balance(tokens, experts, topk, seqs, ld, score, bf16):
    dg = require_gpu()
    rng = np.random.default_rng(tokens + experts)
    raw, x, ids = make(rng, tokens, experts, topk, bf16)
    off = cuts(rng, tokens, seqs)
    n = max(1, seqs)
    tx, tids = on_device(raw, ld), torch.as_tensor(ids, device="cuda")
    toff = None if off is None else torch.as_tensor(off, device="cuda")
    counts, used = torch.full((n, experts), -5, dtype=torch.int32, device="cuda"), torch.full((n,), -5, dtype=torch.int32, device="cuda")
    loss = torch.full((1,), float("nan"), device="cuda")
    ws = workspace(dg.dg_get_moe_balance_workspace_size(tokens, experts, n))
    (dg.dg_moe_balance_bf16 if bf16 else dg.dg_moe_balance)(tx, tids, counts, used, loss, seq_offsets=toff, score=score, coef=0.25, workspace=ws)
    want_counts, want_used, want_loss = block.balance(x, ids, off, score, 0.25)
    assert np.array_equal(host(counts), want_counts) and np.array_equal(host(used), want_used)
    close(host(loss).astype(np.float64), want_loss, want_loss, "loss")
    ws.fill_(0xFF)
    again = torch.zeros(1, device="cuda")
    (dg.dg_moe_balance_bf16 if bf16 else dg.dg_moe_balance)(tx, tids, counts, used, again, seq_offsets=toff, score=score, coef=0.25, workspace=ws)
    assert torch.equal(again, loss)

    bwd = dg.dg_moe_balance_bwd_bf16 if bf16 else dg.dg_moe_balance_bwd
    dloss = torch.full((1,), -1.5, device="cuda")
    want, inside, mag = block.balance_bwd(x, want_counts, want_used, topk, off, score, 0.25, dloss=-1.5)
    half = 2.0 ** -8 if bf16 else 2.0 ** -24
    kind = torch.bfloat16 if bf16 else torch.float32
    whole = torch.full((tokens, ld + 8), 7.0, dtype=kind, device="cuda")
    out = whole[:, :experts]
    bwd(tx, counts, used, out, topk, seq_offsets=toff, dloss=dloss, score=score, coef=0.25)
    got = out.double().cpu().numpy()
    close(got[inside], want[inside], mag[inside], "dlogits", half * np.abs(want[inside]) + (2.0 ** -134 if bf16 else 0))
    assert np.all(got[~inside] == 7.0) and bool((whole[:, experts:] == 7.0).all())
    # With a gradient to add to, beside and in place.
    add = (0.1 * rng.standard_normal((tokens, experts))).astype(np.float32)
    tadd = torch.as_tensor(add, device="cuda").to(kind)
    add = tadd.double().cpu().numpy()
    bwd(tx, counts, used, out, topk, seq_offsets=toff, dloss=dloss, add=tadd, score=score, coef=0.25)
    got = out.double().cpu().numpy()
    sum_ = want + add
    close(got[inside], sum_[inside], mag[inside], "dlogits + add", 2 * half * np.abs(sum_[inside]) + 2.0 ** -24 * np.abs(add[inside]))
    place = tadd.clone()
    bwd(tx, counts, used, place, topk, seq_offsets=toff, dloss=dloss, add=place, score=score, coef=0.25)
    assert torch.equal(place[inside], out[inside]) and torch.equal(place[~inside], tadd[~inside])


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_gradient_against_differences_of_the_loss(score):
    """dlogits against the library's own loss at logits half a unit apart: float32 losses of about coef = 2^20, off
    by at most 2^-16 of it each (2^5 here), and the loss' third derivative along a logit: |d3 p / dx3| <= p, so the
    difference of step h = 1/4 is off by h^2 / 6 of 2 max f p coef / tokens."""
    dg = require_gpu()
    rng = np.random.default_rng(9)
    t, e, k, coef, h = 4, 8, 2, 2.0 ** 20, 0.25
    x = rng.integers(-8, 9, (t, e)).astype(np.float32) / 4
    ids = torch.as_tensor(np.argsort(-x, 1)[:, :k].astype(np.int32).copy(), device="cuda")
    counts, used = torch.zeros(1, e, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = workspace(dg.dg_get_moe_balance_workspace_size(t, e))

    def loss(v):
        out = torch.zeros(1, device="cuda")
        dg.dg_moe_balance(torch.as_tensor(v, device="cuda"), ids, counts, used, out, score=score, coef=coef, workspace=ws)
        return float(out)

    value = loss(x)
    d = torch.zeros(t, e, device="cuda")
    dg.dg_moe_balance_bwd(torch.as_tensor(x, device="cuda"), counts, used, d, k, score=score, coef=coef)
    f = float(counts.max()) * e / (k * t)
    for at in np.ndindex(t, e):
        up, down = x.copy(), x.copy()
        up[at] += h
        down[at] -= h
        got = (loss(up) - loss(down)) / (2 * h)
        assert abs(got - float(d[at])) <= 2.0 ** -16 * value * 2 / h + h * h / 6 * 2 * f * coef / t * 6, (at, got, float(d[at]))


def test_scores_that_leave_float32():
    """Sigmoid scores of -200 and softmax logits of thousands have shares like any other."""
    dg = require_gpu()
    x = np.array([[-200.0, -201.0, -205.0, -300.0], [3000.0, 2999.0, -3000.0, 0.0], [90.0, 85.0, 0.0, -95.0]], dtype=np.float32)
    ids = np.array([[0, 1], [0, 1], [0, 2]], dtype=np.int32)
    for score in ("softmax", "sigmoid"):
        counts, used = torch.zeros(1, 4, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
        loss, d = torch.zeros(1, device="cuda"), torch.zeros(3, 4, device="cuda")
        tx = torch.as_tensor(x, device="cuda")
        dg.dg_moe_balance(tx, torch.as_tensor(ids, device="cuda"), counts, used, loss, score=score,
                          workspace=workspace(dg.dg_get_moe_balance_workspace_size(3, 4)))
        dg.dg_moe_balance_bwd(tx, counts, used, d, 2, score=score)
        c, u, want = block.balance(x, ids, None, score)
        close(host(loss).astype(np.float64), want, want, score)
        grad, _, mag = block.balance_bwd(x, c, u, 2, None, score)
        close(host(d).astype(np.float64), grad, mag, score, 2.0 ** -24 * np.abs(grad))


def test_nan_shows_in_the_loss_and_in_its_own_row():
    dg = require_gpu()
    rng = np.random.default_rng(10)
    x = rng.standard_normal((40, 16)).astype(np.float32)
    x[7, 3] = np.nan
    ids = torch.zeros(40, 1, dtype=torch.int32, device="cuda")
    for score in ("softmax", "sigmoid"):
        counts, used = torch.zeros(1, 16, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
        loss, d = torch.zeros(1, device="cuda"), torch.zeros(40, 16, device="cuda")
        tx = torch.as_tensor(x, device="cuda")
        dg.dg_moe_balance(tx, ids, counts, used, loss, score=score, workspace=workspace(dg.dg_get_moe_balance_workspace_size(40, 16)))
        assert int(used) == 40 and int(counts[0, 0]) == 40 and bool(loss.isnan())
        dg.dg_moe_balance_bwd(tx, counts, used, d, 1, score=score)
        assert bool(d[7].isnan().all()) and bool(d.isnan().sum() == 16)


def test_wild_offsets_stay_in_bounds():
    """Offsets that go down or leave the tokens: results are unspecified, the tokens around are left alone."""
    dg = require_gpu()
    rng = np.random.default_rng(11)
    tokens, experts = 500, 16
    x = torch.randn(tokens, experts, device="cuda")
    ids = torch.zeros(tokens, 2, dtype=torch.int32, device="cuda")
    for trial in range(6):
        off = torch.as_tensor(rng.choice([-2 ** 31, -7, 0, 3, 100, 400, 499, 500, 501, 2 ** 31 - 1], 9).astype(np.int32), device="cuda")
        counts, used = torch.zeros(8, experts, dtype=torch.int32, device="cuda"), torch.zeros(8, dtype=torch.int32, device="cuda")
        loss = torch.zeros(1, device="cuda")
        ws = torch.zeros(dg.dg_get_moe_balance_workspace_size(tokens, experts, 8) + 4096, dtype=torch.uint8, device="cuda")
        ws[-4096:] = 0x77
        dg.dg_moe_balance(x, ids, counts, used, loss, seq_offsets=off, workspace=ws[:-4096])
        whole = torch.full((tokens + 64, experts), 7.0, device="cuda")
        dg.dg_moe_balance_bwd(x, counts, used, whole[32:-32], 2, seq_offsets=off)
        torch.cuda.synchronize()
        assert bool((ws[-4096:] == 0x77).all()) and bool((whole[:32] == 7).all()) and bool((whole[-32:] == 7).all())


def test_more_sequences_than_tokens():
    dg = require_gpu()
    seqs = 70000
    x, ids = torch.randn(3, 8, device="cuda"), torch.tensor([[0, 1], [2, 1], [7, 0]], dtype=torch.int32, device="cuda")
    off = torch.zeros(seqs + 1, dtype=torch.int32, device="cuda")
    off[1000:] = 1
    off[50000:] = 3
    counts, used = torch.full((seqs, 8), -1, dtype=torch.int32, device="cuda"), torch.full((seqs,), -1, dtype=torch.int32, device="cuda")
    loss, d = torch.zeros(1, device="cuda"), torch.zeros(3, 8, device="cuda")
    dg.dg_moe_balance(x, ids, counts, used, loss, seq_offsets=off, coef=seqs, workspace=workspace(dg.dg_get_moe_balance_workspace_size(3, 8, seqs)))
    assert int(used.sum()) == 3 and int(used[999]) == 1 and int(used[49999]) == 2 and int(counts.sum()) == 6 and int(counts.min()) == 0
    few = np.array([0, 1, 3])
    c, u, want = block.balance(x.double().cpu().numpy(), ids.cpu().numpy(), few, coef=2)  # the others add nothing
    close(host(loss).astype(np.float64), want, want, "loss")
    dg.dg_moe_balance_bwd(x, counts, used, d, 2, seq_offsets=off, coef=seqs)
    grad, _, mag = block.balance_bwd(x.double().cpu().numpy(), c, u, 2, few, coef=2)
    close(host(d).astype(np.float64), grad, mag, "dlogits", 2.0 ** -24 * np.abs(grad))


def test_balance_follows_the_router_on_a_stream_and_in_a_graph():
    """Route, balance and both gradients as a training step calls them, replayed with other logits."""
    dg = require_gpu()
    t, e, k = 3000, 64, 4
    gen = torch.Generator(device="cuda").manual_seed(3)
    sets = [torch.randn(t, e, generator=gen, device="cuda") for _ in range(3)]
    x = sets[0].clone()
    ids, w, dw = torch.zeros(t, k, dtype=torch.int32, device="cuda"), torch.zeros(t, k, device="cuda"), torch.randn(t, k, device="cuda")
    counts, used = torch.zeros(1, e, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    loss, d = torch.zeros(1, device="cuda"), torch.zeros(t, e, device="cuda")
    ws = workspace(dg.dg_get_moe_balance_workspace_size(t, e))

    def step():
        dg.dg_moe_route(x, ids, w, score="sigmoid")
        dg.dg_moe_balance(x, ids, counts, used, loss, score="sigmoid", coef=0.01, workspace=ws)
        dg.dg_moe_route_bwd(x, ids, dw, d, score="sigmoid")
        dg.dg_moe_balance_bwd(x, counts, used, d, k, add=d, score="sigmoid", coef=0.01)
        return [v.clone() for v in (counts, used, loss, d)]

    want = []
    for v in sets:
        x.copy_(v)
        want.append(step())
    assert int(want[0][0].sum()) == t * k
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for a, b in zip(step(), want[2]):
            assert torch.equal(a, b)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for i in (0, 2, 1, 0):
        x.copy_(sets[i])
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want[i]):
            assert torch.equal(a, b)
