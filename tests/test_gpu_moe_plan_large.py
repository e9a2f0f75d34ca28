"""GPU row plans (dg_moe_plan_*) of many entries and groups, where the blocks'
counts are added up by a launch of their own, up to the largest size that the
interface takes.  Whole numbers, equal to a stable sort's."""

import pytest
import torch

from tests.gpu_util import require_gpu

pytestmark = pytest.mark.gpu


def _i32(*shape):
    return torch.full(shape, -9, dtype=torch.int32, device="cuda")


def _workspace(dg, tokens, topk, groups):
    size = dg.dg_get_moe_plan_workspace_size(tokens, topk, groups)
    return torch.full((size + 64,), 0xA5, dtype=torch.uint8, device="cuda"), size


def _ranks(g, groups):
    """Rank of each entry in its group (entries with g < 0: no meaning) and the groups' sizes."""
    count = torch.bincount(g[g >= 0], minlength=groups)
    order = torch.where(g >= 0, g, groups).sort(stable=True).indices
    first = torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), count.cumsum(0)])
    rank = torch.empty_like(g)
    rank[order] = torch.arange(g.numel(), device="cuda") - first[torch.where(g >= 0, g, groups)[order]]
    return rank, count


@pytest.mark.parametrize("tokens,topk,experts,first,groups", [
    (2048, 8, 1100, 7, 1024),          # as many counts as blocks x groups from which they are scanned
    (2047, 8, 1024, 0, 1024), (15000, 8, 128, 0, 128), (65409, 2, 200, 3, 130), (131073, 8, 1, 0, 1),
    (131072, 8, 5, 1, 3), (100003, 10, 40, 0, 33), (300000, 7, 256, 0, 256), (40000, 32, 1500, 400, 1000)])
def test_scanned_counts(tokens, topk, experts, first, groups):
    dg = require_gpu()
    gen = torch.Generator(device="cuda")
    gen.manual_seed(tokens)
    ids = torch.randint(-1, experts, (tokens, topk), generator=gen, device="cuda", dtype=torch.int32)
    ids[: tokens // 3] = ids[: tokens // 3] % max(1, experts // 5)  # crowded experts
    g = ids.reshape(-1).long() - first
    g = torch.where((ids.reshape(-1) >= 0) & (g >= 0) & (g < groups), g, -1)
    rank, count = _ranks(g, groups)
    entry = torch.arange(g.numel(), device="cuda")
    ws, size = _workspace(dg, tokens, topk, groups)
    for short in (0, 640):  # room for all, and too little
        ends = ((count + 127) // 128 * 128).cumsum(0)
        total = max(128, int(ends[-1]) - short) if short else int(ends[-1]) + 256
        start = torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), ends])
        row = start[g.clamp(min=0)] + rank
        here = (g >= 0) & (row < total)
        rows, src, m_indices, off = _i32(tokens, topk), _i32(total), _i32(total), _i32(groups + 1)
        dg.dg_moe_plan_contiguous(ids, rows, src, m_indices, off, first_expert=first, workspace=ws)
        assert torch.equal(rows.reshape(-1).long(), torch.where(here, row, -1))
        want = torch.full((total,), -1, dtype=torch.int64, device="cuda")
        want[row[here]] = entry[here]
        assert torch.equal(src.long(), want)
        want[row[here]] = g[here]
        assert torch.equal(m_indices.long(), want)
        assert torch.equal(off.long(), start.clamp(max=total))
    m_max = int(count.max()) * 2 // 3 + 1
    rows, src, used = _i32(tokens, topk), _i32(groups * m_max), _i32(groups)
    dg.dg_moe_plan_masked(ids, rows, src, used, first_expert=first, workspace=ws)
    here = (g >= 0) & (rank < m_max)
    assert torch.equal(rows.reshape(-1).long(), torch.where(here, g * m_max + rank, -1))
    want = torch.full((groups * m_max,), -1, dtype=torch.int64, device="cuda")
    want[(g * m_max + rank)[here]] = entry[here]
    assert torch.equal(src.long(), want)
    assert torch.equal(used.long(), count.clamp(max=m_max))
    assert bool((ws[size:] == 0xA5).all())


def test_most_entries_and_groups():
    """2^31 - 32 entries of 1024 groups: 2^31 counts, indexed with 64 bits.  Entry i is
    of expert i mod 1000, so that its rank is i / 1000; the last rows do not fit."""
    dg = require_gpu()
    topk, groups, experts = 32, 1024, 1000
    tokens = 2 ** 26 - 1
    entries, total = tokens * topk, 2 ** 31 - 128
    ids = torch.empty(tokens, topk, dtype=torch.int32, device="cuda")
    flat, step = ids.view(-1), 1 << 27
    for lo in range(0, entries, step):
        flat[lo:lo + step] = torch.arange(lo, min(lo + step, entries), device="cuda") % experts
    rows, src, m_indices, off = _i32(tokens, topk), _i32(total), _i32(total), _i32(groups + 1)
    ws = torch.empty(dg.dg_get_moe_plan_workspace_size(tokens, topk, groups), dtype=torch.uint8, device="cuda")
    dg.dg_moe_plan_contiguous(ids, rows, src, m_indices, off, workspace=ws)
    count = torch.tensor([(entries - g + experts - 1) // experts if g < experts else 0 for g in range(groups)], device="cuda")
    start = torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), ((count + 127) // 128 * 128).cumsum(0)])
    assert int(start[-1]) > total  # some are dropped
    assert torch.equal(off.long(), start.clamp(max=total))
    kept = 0
    for lo in range(0, entries, step):
        i = torch.arange(lo, min(lo + step, entries), device="cuda")
        row = start[i % experts] + i // experts
        row = torch.where(row < total, row, -1)
        assert torch.equal(rows.view(-1)[lo:lo + step].long(), row)
        i, row = i[row >= 0], row[row >= 0]
        kept += i.numel()
        assert torch.equal(src[row].long(), i) and torch.equal(m_indices[row].long(), i % experts)
        del i, row
    assert int((src >= 0).sum()) == kept and int((m_indices >= 0).sum()) == kept
