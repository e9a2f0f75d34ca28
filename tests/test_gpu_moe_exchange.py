"""GPU exchange between token rows and expert rows (dg_moe_plan_*,
dg_moe_dispatch*, dg_moe_combine, dg_moe_combine_bwd) against oracle/moe.py
and the oracle's quantisers.

Plans are whole numbers and must be equal; dispatched codes and scales equal
the activation quantiser's bit for bit; combined rows are held to one bf16
rounding (2^-8) and 2^-22 of the sum of the terms' magnitudes for the float32
sum; gradient codes must be a nearest e4m3 number of v / s for a v / s within
2^-18 of the oracle's, scales within 2^-20.
"""

import numpy as np
import pytest
import torch

import synth
from oracle import e4m3, moe, quant, ue8m0
from tests.gpu_util import bf16_to_f64, dev, host, require_gpu

pytestmark = pytest.mark.gpu

FILL = 0x5A  # what unwritten codes keep


def _i32(*shape, value=-9):
    return torch.full(shape, value, dtype=torch.int32, device="cuda")


def make_ids(rng, tokens, topk, experts, dropped=0.1):
    ids = np.array([rng.permutation(experts)[:topk] for _ in range(tokens)], dtype=np.int32).reshape(tokens, topk)
    ids[rng.random(ids.shape) < dropped] = -1
    return ids


def gpu_plan(dg, ids, first, groups, m_total=None, m_max=None):
    tokens, topk = ids.shape
    ws = torch.full((max(16, dg.dg_get_moe_plan_workspace_size(tokens, topk, groups)),), 0xA5, dtype=torch.uint8, device="cuda")
    rows = _i32(tokens, topk)
    t = torch.as_tensor(ids, device="cuda")
    if m_max is not None:
        src, count = _i32(groups * m_max), _i32(groups)
        dg.dg_moe_plan_masked(t, rows, src, count, first_expert=first, workspace=ws)
        return rows, src, count
    src, m_indices, off = _i32(m_total), _i32(m_total), _i32(groups + 1)
    dg.dg_moe_plan_contiguous(t, rows, src, m_indices, off, first_expert=first, workspace=ws)
    return rows, src, m_indices, off


PLANS = [  # tokens, topk, experts, first, groups, contiguous rows, masked rows
    (0, 2, 4, 0, 4, 256, 8), (1, 1, 1, 0, 1, 128, 1), (1, 8, 256, 0, 256, 1024, 4), (7, 3, 9, 4, 3, 512, 5),
    (128, 8, 256, 64, 32, 4096, 128), (1000, 4, 16, 0, 16, 6144, 300), (1000, 4, 16, 12, 4, 640, 100),
    (5000, 8, 40, 8, 8, 9216, 1024), (9001, 2, 1024, 0, 1024, 131072, 16), (300, 32, 33, 1, 32, 0, 0),
    (20011, 6, 6, 2, 1, 20096, 20011), (100, 4, 64, 0, 64, 262144, 8192)]


@pytest.mark.parametrize("case", PLANS, ids=str)
def test_plan(case):
    dg = require_gpu()
    tokens, topk, experts, first, groups, m_total, m_max = case
    ids = make_ids(np.random.default_rng(tokens + topk), tokens, topk, experts)
    for got, ref in ((gpu_plan(dg, ids, first, groups, m_total=m_total), moe.plan_contiguous(ids, first, groups, m_total)),
                     (gpu_plan(dg, ids, first, groups, m_max=m_max), moe.plan_masked(ids, first, groups, m_max))):
        for a, b in zip(got, ref):
            assert np.array_equal(a.cpu().numpy(), b)


def test_plan_with_ids_out_of_range():
    dg = require_gpu()
    rng = np.random.default_rng(1)
    ids = rng.choice(np.array([-2**31, -1, 0, 3, 4, 5, 6, 7, 2**31 - 1], dtype=np.int32), (500, 3))
    got, ref = gpu_plan(dg, ids, 4, 3, m_total=1024), moe.plan_contiguous(ids, 4, 3, 1024)
    for a, b in zip(got, ref):
        assert np.array_equal(a.cpu().numpy(), b)
    got = gpu_plan(dg, ids, 2**31 - 1, 3, m_max=64)
    for a, b in zip(got, moe.plan_masked(ids, 2**31 - 1, 3, 64)):
        assert np.array_equal(a.cpu().numpy(), b)


@pytest.mark.parametrize("skew", [0, 1, 2])
def test_plan_with_crowded_experts(skew):
    """All entries on one expert, on none, or on the first and last."""
    dg = require_gpu()
    ids = np.full((3000, 4), [5, -1, 0][skew], dtype=np.int32)
    if skew == 2:
        ids[:, 1:] = 7
    got, ref = gpu_plan(dg, ids, 0, 8, m_total=12160), moe.plan_contiguous(ids, 0, 8, 12160)
    for a, b in zip(got, ref):
        assert np.array_equal(a.cpu().numpy(), b)


def _dispatch(dg, x, src, topk, groups, rows, ue8m0_scales, pad_x=0, ld_sf=None):
    cols = x.shape[1]
    t = dev(np.pad(x, ((0, 0), (0, pad_x)))) if pad_x else dev(x)
    t = t[:, :cols]
    ld = (rows + 3) // 4 * 4 if ld_sf is None else ld_sf
    shape = (groups,) if groups > 1 else ()
    q = torch.full((*shape, rows, cols), FILL, dtype=torch.uint8, device="cuda")
    sf = torch.full((*shape, cols // 128, ld), 0x5A if ue8m0_scales else -3.0, dtype=torch.uint8 if ue8m0_scales else torch.float32,
                    device="cuda")
    (dg.dg_moe_dispatch_ue8m0 if ue8m0_scales else dg.dg_moe_dispatch)(t, torch.as_tensor(src, device="cuda"), q, sf, topk=topk)
    return host(q).reshape(groups, rows, cols), host(sf).reshape(groups, cols // 128, ld)


@pytest.mark.parametrize("ue", [False, True])
@pytest.mark.parametrize("tokens,topk,cols,groups,rows,pad,ld", [
    (1, 1, 128, 1, 128, 0, None), (5, 3, 256, 1, 256, 8, 260), (130, 8, 1152, 4, 37, 0, 44), (700, 2, 7168, 1, 2304, 0, None),
    (3000, 6, 128, 1, 18432, 16, None), (64, 8, 384, 32, 16, 0, None)])
def test_dispatch(ue, tokens, topk, cols, groups, rows, pad, ld):
    dg = require_gpu()
    rng = np.random.default_rng(cols + rows)
    x = synth.bf16_normal((tokens, cols), 77)
    x[0, :128] = 0  # an all-zero tile
    src = np.full(groups * rows, -1, dtype=np.int32)
    use = rng.random(src.size) < 0.7
    src[use] = rng.integers(0, tokens * topk, int(use.sum()))
    src[::11] = tokens * topk + rng.integers(0, 5, src[::11].size)  # names no entry
    src[1::13] = -2**31
    if src.size > 2:
        src[2] = 0
    q, sf = _dispatch(dg, x, src, topk, groups, rows, ue, pad, ld)
    ref_q, ref_sf = (ue8m0.quant_1x128_ue8m0 if ue else quant.quant_1x128)(x)
    live = (src >= 0) & (src < tokens * topk)
    token = np.where(live, src // topk, 0)
    flat = q.reshape(-1, cols)
    assert np.array_equal(flat[live], ref_q[token[live]]) and np.all(flat[~live] == FILL)
    for g in range(groups):
        part = slice(g * rows, (g + 1) * rows)
        want = np.where(live[part], ref_sf[:, token[part]], np.array(0x5A if ue else -3.0, dtype=ref_sf.dtype))
        assert np.array_equal(sf[g][:, :rows], want)
        assert np.all(sf[g][:, rows:] == (0x5A if ue else -3.0))


def test_dispatch_every_tile_maximum():
    """One tile for every positive finite bf16 as its largest magnitude, the
    others below it in magnitude, zeros of both signs among them."""
    dg = require_gpu()
    amax = np.arange(1, 0x7F80, dtype=np.uint16)
    rng = np.random.default_rng(3)
    x = (rng.random((amax.size, 128)) * (amax[:, None] + 1)).astype(np.uint16)
    near = rng.random(x.shape) < 0.5  # half of them in the few binades that do not become zero
    x = np.where(near, np.maximum(amax[:, None].astype(np.int64) - rng.integers(0, 1800, x.shape), 0).astype(np.uint16), x)
    x |= (rng.integers(0, 2, x.shape) << 15).astype(np.uint16)
    x[:, 0] = amax
    x[:, 1], x[:, 2] = 0x0000, 0x8000
    for ue in (False, True):
        q, sf = _dispatch(dg, x, np.arange(amax.size, dtype=np.int32), 1, 1, amax.size, ue)
        ref_q, ref_sf = (ue8m0.quant_1x128_ue8m0 if ue else quant.quant_1x128)(x)
        assert np.array_equal(sf[0][:, :amax.size], ref_sf[:, :amax.size])
        assert np.array_equal(q[0], ref_q)


@pytest.mark.parametrize("weighted", [True, False])
@pytest.mark.parametrize("tokens,topk,cols,total,pad", [
    (1, 1, 8, 1, 0), (3, 2, 136, 5, 8), (100, 8, 2048, 300, 0), (65, 32, 2056, 64, 16), (40, 6, 7168, 0, 0), (513, 3, 4104, 999, 0)])
def test_combine(weighted, tokens, topk, cols, total, pad):
    dg = require_gpu()
    rng = np.random.default_rng(tokens + cols)
    d = synth.bf16_normal((max(total, 1), cols), 78)[:total]
    rows = rng.integers(-1, max(total, 1), (tokens, topk)).astype(np.int32)
    rows[rng.random(rows.shape) < 0.2] = total
    rows[0] = -1
    w = rng.random((tokens, topk)).astype(np.float32) if weighted else None
    td = dev(np.pad(d, ((0, 0), (0, pad))))[:, :cols]
    y = torch.full((tokens, cols + pad), 3.0, dtype=torch.bfloat16, device="cuda")
    dg.dg_moe_combine(td, torch.as_tensor(rows, device="cuda"), y[:, :cols], weights=None if w is None else torch.as_tensor(w, device="cuda"))
    got = bf16_to_f64(host(y))
    ref, size = moe.combine(bf16_to_f64(d), rows, w)
    assert np.all(np.abs(got[:, :cols] - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -22 * topk * size)
    assert np.all(got[0, :cols] == 0) and np.all(got[:, cols:] == 3.0)


def test_combine_does_not_read_unnamed_rows():
    dg = require_gpu()
    d = np.full((4, 256), 0x7FC0, dtype=np.uint16)  # NaN
    d[2] = synth.bf16_normal((256,), 5)
    rows = torch.tensor([[2, -1], [-1, -1], [4, 2]], dtype=torch.int32, device="cuda")
    y = torch.empty(3, 256, dtype=torch.bfloat16, device="cuda")
    dg.dg_moe_combine(dev(d), rows, y)
    got = host(y)
    assert np.array_equal(got[0], d[2]) and np.array_equal(got[2], d[2]) and np.all(got[1] == 0)


def check_codes(q, s, v, ref_s, live, what):
    """Codes q and scales s (broadcast over the last axis: one a value) of the
    oracle's values v with scales ref_s."""
    assert np.all(np.abs(s - ref_s) <= 2.0 ** -20 * ref_s), what
    t = np.where(ref_s > 0, v / np.where(ref_s > 0, ref_s, 1.0), 0.0)
    off = np.abs(e4m3.decode(q).astype(np.float64) - t)
    ok = off <= moe.half_step(np.abs(t) * (1 + 2.0 ** -18)) + 2.0 ** -18 * np.abs(t)
    assert np.all(ok[live]), what


@pytest.mark.parametrize("transposed", [True, False])
@pytest.mark.parametrize("tokens,topk,experts,first,groups,cols,m_total", [
    (1, 1, 1, 0, 1, 128, 128), (50, 3, 6, 1, 4, 256, 640), (333, 8, 16, 4, 4, 1152, 1280), (300, 2, 4, 0, 4, 384, 256),
    (9, 2, 4, 0, 4, 128, 0)])
def test_combine_bwd(transposed, tokens, topk, experts, first, groups, cols, m_total):
    dg = require_gpu()
    rng = np.random.default_rng(cols + tokens)
    ids = make_ids(rng, tokens, topk, experts)
    rows, src, _, _ = gpu_plan(dg, ids, first, groups, m_total=m_total)
    dy, d = synth.bf16_normal((tokens, cols), 80), synth.bf16_normal((max(m_total, 1), cols), 81)[:m_total]
    dy[0, :128] = 0
    w = rng.random((tokens, topk)).astype(np.float32)
    d[src.cpu().numpy() < 0] = 0x7FC0  # rows not in use are not looked at
    dq = torch.full((m_total, cols), FILL, dtype=torch.uint8, device="cuda")
    dsf = torch.full((cols // 128, m_total + 4), -3.0, device="cuda")
    dqt = torch.full((cols, m_total), FILL, dtype=torch.uint8, device="cuda") if transposed else None
    dsft = torch.full((m_total // 128, cols + 8), -3.0, device="cuda") if transposed else None
    dw = torch.full((tokens, topk), float("nan"), device="cuda")
    ws = torch.full((max(16, dg.dg_get_moe_combine_bwd_workspace_size(m_total, cols)),), 0xFF, dtype=torch.uint8, device="cuda")
    dg.dg_moe_combine_bwd(dev(dy), dev(d), src, rows, torch.as_tensor(w, device="cuda"), dq, dsf, dqt, dsft, dw, workspace=ws)
    src, rows = src.cpu().numpy(), rows.cpu().numpy()
    ref, ref_dw, size = moe.combine_bwd(bf16_to_f64(dy), bf16_to_f64(d), src, rows, w)
    live = src >= 0
    # float32 sums of `cols` products
    assert np.all(np.abs(dw.cpu().numpy() - ref_dw) <= 2.0 ** -24 * 64 * size + 1e-30)
    if m_total == 0:
        return
    rs = moe.row_scales(ref)
    dsf = host(dsf)
    assert np.all(dsf[:, :m_total][:, ~live] == -3.0) and np.all(dsf[:, m_total:] == -3.0)
    q = host(dq)
    assert np.all(q[~live] == FILL)
    check_codes(q[live], np.repeat(dsf[:, :m_total].T, 128, axis=1)[live], ref[live], np.repeat(rs.T, 128, axis=1)[live],
                slice(None), "rows")
    if transposed:
        check_transposed(host(dqt), host(dsft), ref, live, cols)


@pytest.mark.parametrize("transposed", [True, False])
def test_combine_bwd_tall(transposed):
    """A layout above the size up to which the weights' gradient is summed apart from the tiles."""
    test_combine_bwd(transposed, 13000, 3, 4, 1, 3, 512, 41088)


def test_combine_bwd_many_entries():
    """More entries than are summed apart from the tiles, most of them without a row."""
    test_combine_bwd(True, 8300, 4, 64, 3, 2, 256, 1536)


def check_transposed(qt, sft, v, live, cols):
    blocks = live.reshape(-1, 128).any(1)
    rows = np.repeat(blocks, 128)
    assert np.all(qt[:, ~rows] == FILL) and np.all(sft[~blocks] == -3.0) and np.all(sft[:, cols:] == -3.0)
    assert np.all(e4m3.decode(qt[:, rows & ~live]) == 0)
    cs = moe.column_scales(v)
    check_codes(qt.T[rows], np.repeat(sft[:, :cols], 128, axis=0)[rows], v[rows], np.repeat(cs, 128, axis=0)[rows],
                live[rows], "columns")


def test_large_offsets():
    """Layouts past 2^32 bytes: rows near the end are addressed with 64 bits."""
    dg = require_gpu()
    cols, total, tokens = 7168, 614400, 64  # 4.4 GB of codes, 8.8 GB of bf16 rows
    x = synth.bf16_normal((tokens, cols), 90)
    src = torch.full((total,), -1, dtype=torch.int32, device="cuda")
    at = torch.arange(total - 3 * tokens, total, 3, device="cuda")
    src[at] = torch.arange(tokens, dtype=torch.int32, device="cuda")
    q = torch.zeros((total, cols), dtype=torch.uint8, device="cuda")
    sf = torch.zeros((cols // 128, total), device="cuda")
    dg.dg_moe_dispatch(dev(x), src, q, sf, topk=1)
    ref_q, ref_sf = quant.quant_1x128(x)
    assert np.array_equal(host(q[at]), ref_q) and np.array_equal(host(sf[:, at]), ref_sf[:, :tokens])
    assert int(q[:total - 3 * tokens].view(torch.int64).ne(0).sum()) == 0
    del q
    d = torch.zeros((total, cols), dtype=torch.bfloat16, device="cuda")
    d.view(torch.int16)[at] = dev(x)
    y = torch.empty(tokens, cols, dtype=torch.bfloat16, device="cuda")
    dg.dg_moe_combine(d, at.to(torch.int32).view(-1, 1), y)
    assert np.array_equal(host(y), x)
