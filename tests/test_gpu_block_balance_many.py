"""GPU load balance of a router over so many tokens that a wave adds up many of them,
against 64 bits on the device.

A chunk is a 256th of the tokens and has 16 waves, each of which adds the float32 shares of
its tokens one after another: n = tokens / 4096 additions, each within 2^-24 of the sum so
far, all positive.  Behind them the 16 waves and up to 256 chunks are added (at most 16 + 32
additions in a row), and the products with f (64 lanes, 16 workgroups, 8 roundings): 2^-18.
A share is within 2^-17 of itself (tests/test_gpu_block_balance.py); the loss is positive.
"""

import numpy as np
import pytest
import torch

from tests.block_util import workspace
from tests.gpu_util import require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def release():
    yield
    torch.cuda.empty_cache()


def bound(tokens):
    return (-(-tokens // 4096)) * 2.0 ** -24 + 2.0 ** -18 + 2.0 ** -17


def exact(logits, ids, ends, score, coef):
    """(counts, used, loss) in 64 bits, 16384 tokens at a time."""
    experts, topk, seqs = logits.shape[1], ids.shape[1], len(ends) - 1
    counts, used, loss = [], [], 0.0
    for a, b in zip(ends[:-1], ends[1:]):
        total, chosen, n = torch.zeros(experts, dtype=torch.float64, device="cuda"), torch.zeros(experts + 1, dtype=torch.int64, device="cuda"), 0
        for at in range(a, b, 16384):
            part = slice(at, min(at + 16384, b))
            x = logits[part].double()
            live = ~torch.isneginf(x).all(1)
            x = x[live]
            p = torch.softmax(x, 1) if score == "softmax" else torch.sigmoid(x) / torch.sigmoid(x).sum(1, keepdim=True)
            total += p.sum(0)
            here = ids[part][live].long().flatten()
            chosen += torch.bincount(torch.where((here >= 0) & (here < experts), here, experts), minlength=experts + 1)
            n += int(live.sum())
        counts.append(chosen[:experts])
        used.append(n)
        if n:
            loss += float((experts * chosen[:experts].double() / (topk * n) * total).sum()) / n
    return torch.stack(counts).int(), used, coef * loss / seqs


def check(tokens, experts, topk, cuts, score, kind, seed):
    dg = require_gpu()
    g = torch.Generator(device="cuda").manual_seed(seed)
    part = 2 * torch.randn(min(tokens, 65521), experts, generator=g, device="cuda") + torch.randn(1, experts, generator=g, device="cuda")
    part[5::97] = -float("inf")
    part[3::11, ::7] = -float("inf")
    logits = part.to(kind).repeat(-(-tokens // len(part)), 1)[:tokens].contiguous()
    del part
    ids = torch.randint(-1, experts, (tokens, topk), generator=g, dtype=torch.int32, device="cuda")
    ends = [0, *cuts, tokens]
    off = torch.tensor(ends, dtype=torch.int32, device="cuda") if cuts else None
    n = len(ends) - 1
    counts, used = torch.zeros(n, experts, dtype=torch.int32, device="cuda"), torch.zeros(n, dtype=torch.int32, device="cuda")
    loss = torch.zeros(1, device="cuda")
    ws = workspace(dg.dg_get_moe_balance_workspace_size(tokens, experts, n))
    (dg.dg_moe_balance if kind == torch.float32 else dg.dg_moe_balance_bf16)(logits, ids, counts, used, loss, seq_offsets=off, score=score, coef=0.5,
                                                                            workspace=ws)
    want_counts, want_used, want = exact(logits, ids, ends, score, 0.5)
    assert torch.equal(counts, want_counts) and used.tolist() == want_used
    assert abs(float(loss) - want) <= bound(tokens) * want, (float(loss), want)
    return abs(float(loss) - want) / want


@pytest.mark.parametrize("tokens,experts,topk,cuts", [(32768, 256, 8, []), (65536, 64, 6, [1, 40000]), (50001, 72, 4, [7, 49000, 49001]), (200000, 130, 2, [])],
                         ids=str)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16])
def test_loss_of_many_tokens(tokens, experts, topk, cuts, score, kind):
    check(tokens, experts, topk, cuts, score, kind, tokens)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_loss_of_more_than_4_gib(score):
    check(1200 * 1024, 1024, 2, [1200 * 1024 - 256], score, torch.float32, 5)


@pytest.mark.parametrize("tokens,topk,cuts", [(3001, 3, []), (3001, 3, [7, 7, 1000, 2990]), (20000, 6, [3, 19998]), (40001, 5, [])], ids=str)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_loss_is_rounded_once(tokens, topk, cuts, score):
    """Equal logits of 0 among a power of two of experts: shares and their sums are exact, and the loss is coef times
    the mean of what part of the choices name an expert, within half a step."""
    dg = require_gpu()
    experts, rng = 64, np.random.default_rng(tokens + len(cuts))
    logits = torch.zeros(tokens, experts, device="cuda")
    ends = [0, *cuts, tokens]
    n = len(ends) - 1
    off = torch.tensor(ends, dtype=torch.int32, device="cuda") if cuts else None
    counts, used = torch.zeros(n, experts, dtype=torch.int32, device="cuda"), torch.zeros(n, dtype=torch.int32, device="cuda")
    loss, ws = torch.zeros(1, device="cuda"), workspace(dg.dg_get_moe_balance_workspace_size(tokens, experts, n))
    for trial in range(12):
        ids = rng.integers(-1 - trial, experts, (tokens, topk)).astype(np.int32)
        coef = float(np.float32(rng.uniform(0.001, 2.0)))
        dg.dg_moe_balance(logits, torch.as_tensor(ids, device="cuda"), counts, used, loss, seq_offsets=off, score=score, coef=coef, workspace=ws)
        want = coef * np.mean([(ids[a:b] >= 0).mean() if b > a else 0.0 for a, b in zip(ends[:-1], ends[1:])])
        assert abs(float(loss) - want) <= 2.0 ** -24 * (1 + 2.0 ** -20) * want, (trial, float(loss), want)
