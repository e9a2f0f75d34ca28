"""GPU mixture-of-experts calls along paths that small shapes do not take."""

import numpy as np
import pytest
import torch

import synth
from oracle import e4m3, moe, quant
from tests.gpu_util import bf16_to_f64, dev, host, require_gpu
from tests.test_gpu_moe_ckpt import make_h
from tests.test_gpu_moe_exchange import FILL, check_codes, check_transposed

pytestmark = pytest.mark.gpu


def _u8(*shape):
    return torch.full(shape, FILL, dtype=torch.uint8, device="cuda")


def _f32(*shape):
    return torch.full(shape, -3.0, device="cuda")


def test_combine_bwd_leaves_blocks_of_rows_that_name_no_entry():
    """Values of src past the entries name no row, like -1: a block of them is not written."""
    dg = require_gpu()
    tokens, topk, cols, m_total = 20, 2, 256, 384
    src = np.full(m_total, tokens * topk + 3, dtype=np.int32)
    src[:40] = np.arange(40)
    src[256:] = np.int32(2 ** 31 - 1)
    src[300] = -5
    rows = np.arange(40, dtype=np.int32).reshape(tokens, topk)
    dy, d = synth.bf16_normal((tokens, cols), 70), synth.bf16_normal((m_total, cols), 71)
    w = np.random.default_rng(1).random((tokens, topk)).astype(np.float32)
    dq, dsf, dqt, dsft = _u8(m_total, cols), _f32(2, m_total), _u8(cols, m_total), _f32(3, cols)
    dw = torch.full((tokens, topk), float("nan"), device="cuda")
    ws = torch.empty(dg.dg_get_moe_combine_bwd_workspace_size(m_total, cols), dtype=torch.uint8, device="cuda")
    dg.dg_moe_combine_bwd(dev(dy), dev(d), torch.as_tensor(src, device="cuda"), torch.as_tensor(rows, device="cuda"),
                          torch.as_tensor(w, device="cuda"), dq, dsf, dqt, dsft, dw, workspace=ws)
    live = np.arange(m_total) < 40
    ref, _, _ = moe.combine_bwd(bf16_to_f64(dy), bf16_to_f64(d), np.where(live, src, -1), rows, w)
    assert np.all(host(dq)[~live] == FILL)
    check_transposed(host(dqt), host(dsft), ref, live, cols)


# ------------------------------------------------------------------ routing --

@pytest.mark.parametrize("groups,keep,group_top", [(1, 1, 2), (4, 2, 2), (4, 2, 1), (8, 3, 2), (16, 5, 2)])
def test_infinite_biases(groups, keep, group_top):
    """A bias of -inf masks its expert like a logit of -inf, one of +inf puts it first."""
    dg = require_gpu()
    rng = np.random.default_rng(groups)
    x = np.stack([rng.permutation(16) * 0.25 - 2.0 for _ in range(40)]).astype(np.float32)
    bias = np.zeros(16, dtype=np.float32)
    bias[[1, 2, 3, 8, 13]], bias[6] = -np.inf, np.inf
    ids, w = torch.empty(40, 4, dtype=torch.int32, device="cuda"), torch.empty(40, 4, device="cuda")
    dg.dg_moe_route(torch.as_tensor(x, device="cuda"), ids, w, bias=torch.as_tensor(bias, device="cuda"), score="sigmoid",
                    expert_groups=groups, topk_groups=keep, group_top=group_top)
    ref, ref_w = moe.route(x, 4, "sigmoid", bias, groups, keep, group_top)
    assert np.array_equal(host(ids), ref) and np.all(ref[:, 0] == 6) and not np.isin(ref, [1, 2, 3, 8, 13]).any()
    assert np.all(np.abs(host(w) - ref_w) <= 2.0 ** -18 * ref_w)


# ------------------------------------------------------- the unit's backward --

def _used(m_total, seed, empty):
    """m_indices with partly filled blocks, and blocks without a row in use at `empty`."""
    rng = np.random.default_rng(seed)
    m = np.full(m_total, -1, dtype=np.int32)
    for b in range(m_total // 128):
        if b not in empty:
            m[b * 128:b * 128 + (128 if rng.random() < 0.6 else rng.integers(1, 129))] = b % 3
    return m


def _bwd_outputs(m_total, inter, with_act):
    out = dict(dq=_u8(m_total, 2 * inter), dsf=_f32(inter // 64, m_total), dqt=_u8(2 * inter, m_total),
               dsft=_f32(m_total // 128, 2 * inter))
    return out | (dict(aqt=_u8(inter, m_total), asft=_f32(m_total // 128, inter)) if with_act else {})


def _same_as_block_alone(dg, hq, hsf, da, m, out, block):
    """Outputs of a block of 128 rows, bit for bit those of a call on its rows alone."""
    rows, inter = slice(block * 128, block * 128 + 128), da.shape[1]
    one = _bwd_outputs(128, inter, "aqt" in out)
    dg.dg_swiglu_bwd(hq[rows], hsf[:, rows].contiguous(), da[rows], None if m is None else m[rows], **one)
    for name, got in out.items():
        part = {"dq": got[rows], "dsf": got[:, rows], "dqt": got[:, rows], "aqt": got[:, rows],
                "dsft": got[block:block + 1], "asft": got[block:block + 1]}[name]
        assert torch.equal(part, one[name]), (name, block)


@pytest.mark.parametrize("with_act", [True, False])
@pytest.mark.parametrize("blocks,inter,mask", [(131, 640, True), (20, 2048, True), (67, 512, False), (300, 128, True), (257, 128, False)])
def test_swiglu_bwd_of_more_tiles_than_workgroups(blocks, inter, mask, with_act):
    """320 to 655 tiles: workgroups take several, of unequal numbers, past unused blocks
    at both ends, alone, and in runs in the middle."""
    dg = require_gpu()
    m_total = blocks * 128
    empty = {0, 1, 5, blocks // 2, blocks // 2 + 1, blocks // 2 + 2, blocks - 1}
    m = _used(m_total, blocks, empty) if mask else None
    live = m >= 0 if mask else np.ones(m_total, dtype=bool)
    hq, hsf = quant.quant_1x128(make_h(m_total, inter, 97))
    hsf = np.ascontiguousarray(hsf[:, :m_total])
    da = synth.bf16_normal((m_total, inter), 98)
    hq[~live], da[~live] = 0x7F, 0x7FC0
    hsf[:, ~live] = np.nan
    tm = None if m is None else torch.as_tensor(m, device="cuda")
    thq, thsf, tda = dev(hq), dev(hsf), dev(da)
    out = _bwd_outputs(m_total, inter, with_act)
    dg.dg_swiglu_bwd(thq, thsf, tda, tm, **out)
    for block in range(blocks):
        _same_as_block_alone(dg, thq, thsf, tda, tm, out, block)
    if inter * blocks <= 41000:  # and the oracle's, where it takes little
        h = np.where(live[:, None], moe.dequant_rows(np.where(live[:, None], hq, 0), np.nan_to_num(hsf)), 0.0)
        dh = np.where(live[:, None], moe.swiglu_bwd(h, bf16_to_f64(np.where(live[:, None], da, 0))), 0.0)
        check_transposed(host(out["dqt"]), host(out["dsft"]), dh, live, 2 * inter)
        s = host(out["dsf"])
        check_codes(host(out["dq"])[live], np.repeat(s.T, 128, axis=1)[live], dh[live],
                    np.repeat(moe.row_scales(dh).T, 128, axis=1)[live], slice(None), "rows")
        if with_act:
            check_transposed(host(out["aqt"]), host(out["asft"]), moe.swiglu(h), live, inter)


def test_swiglu_bwd_large_offsets():
    """More than 2^32 bytes of checkpoint, gradient and transposed codes, few rows in use."""
    dg = require_gpu()
    m_total, inter, used = 614400, 3584, (0, 2399, 4798, 4799)
    m = torch.full((m_total,), -1, dtype=torch.int32, device="cuda")
    hq = torch.full((m_total, 2 * inter), 0x7F, dtype=torch.uint8, device="cuda")
    hsf = torch.full((inter // 64, m_total), float("nan"), device="cuda")
    da = torch.full((m_total, inter), float("nan"), dtype=torch.bfloat16, device="cuda")
    for n, b in enumerate(used):
        rows = slice(b * 128, b * 128 + 128)
        q, sf = quant.quant_1x128(make_h(128, inter, 100 + n))
        hq[rows], hsf[:, rows] = dev(q), dev(sf[:, :128])
        da.view(torch.int16)[rows] = dev(synth.bf16_normal((128, inter), 110 + n))
        m[b * 128:b * 128 + 128 - 5 * n] = n
    out = _bwd_outputs(m_total, inter, True)
    dg.dg_swiglu_bwd(hq, hsf, da, m, **out)
    for b in used:
        _same_as_block_alone(dg, hq, hsf, da, m, out, b)
    for b in (1, 2398, 2400, 4797):
        assert bool((out["dq"][b * 128:b * 128 + 128] == FILL).all()) and bool((out["dqt"][:, b * 128:b * 128 + 128] == FILL).all())
    assert int((out["dsf"] != -3.0).any(0).sum()) == int((m >= 0).sum())
    assert int((out["dsft"] != -3.0).any(1).sum()) == len(used) == int((out["asft"] != -3.0).any(1).sum())


# -------------------------------------------------------------- gated unit --

def _e8(*shape):
    return torch.full(shape, 0x5A, dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("rows,inter,tail", [(1, 128, 0), (37, 256, 0), (640, 1152, 2), (256, 2048, 1)])
def test_swiglu_quant_ue8m0_contiguous(rows, inter, tail):
    dg = require_gpu()
    h = make_h(rows, inter, 121)
    m = np.where(np.random.default_rng(rows).random(rows) < 0.8, 1, -1).astype(np.int32)
    m[0] = 0
    m[rows - 128 * tail:rows if tail else 0] = -1
    live = m >= 0
    h[~live] = 0x7FC0
    ld = (rows + 3) // 4 * 4 + 4
    q, sf = _u8(rows, inter), _e8(inter // 128, ld)
    dg.dg_swiglu_quant_ue8m0(dev(h), q, sf, m_indices=torch.as_tensor(m, device="cuda"))
    q, sf = host(q), host(sf)
    assert np.all(q[~live] == FILL) and np.all(sf[:, :rows][:, ~live] == 0x5A) and np.all(sf[:, rows:] == 0x5A)
    v = moe.swiglu(bf16_to_f64(h[live]))
    amax = np.abs(v).reshape(len(v), -1, 128).max(2).T
    got = sf[:, :rows][:, live].astype(np.int64)
    exact = np.log2(np.where(amax > 0, amax, 448.0) / 448.0)
    e = np.where(amax > 0, np.clip(np.ceil(exact), -127, 127) + 127, 0).astype(np.int64)
    near = np.abs(exact - np.round(exact)) < 2.0 ** -20  # the float32 maximum may fall on either side of a power of two
    assert np.all((got == e) | (near & (np.abs(got - e) <= 1)))
    t = v / np.repeat(np.ldexp(1.0, got - 127).T, 128, axis=1)
    off = np.abs(e4m3.decode(q[live]).astype(np.float64) - t)
    assert np.all(off <= moe.half_step(np.abs(t) * (1 + 2.0 ** -18)) + 2.0 ** -18 * np.abs(t))


@pytest.mark.parametrize("form", ["fp32", "checkpoint", "ue8m0", "masked"])
def test_swiglu_quant_of_more_values_than_the_caches_hold(form):
    """More than 2^25 values are stored past the caches: the same bits as calls on parts of the rows."""
    dg = require_gpu()
    groups, rows, inter = (4, 4208, 2048) if form == "masked" else (1, 16640, 2048)
    h = torch.randn(groups, rows, 2 * inter, generator=torch.Generator(device="cuda").manual_seed(5), device="cuda").bfloat16()
    m = torch.where(torch.arange(rows, device="cuda") % 7 == 3, -1, 0).to(torch.int32)
    count = torch.tensor([rows, 0, 1000, rows + 9], dtype=torch.int32, device="cuda")
    new_sf = _e8 if form == "ue8m0" else _f32
    run = dg.dg_swiglu_quant_ue8m0 if form == "ue8m0" else dg.dg_swiglu_quant

    def call(lo, hi):
        n = hi - lo
        q, sf = _u8(groups, n, inter), new_sf(groups, inter // 128, n)
        more = dict(hq=_u8(n, 2 * inter), hsf=_f32(inter // 64, n)) if form == "checkpoint" else {}
        part = h[:, lo:hi].contiguous()
        if form == "masked":
            run(part, q, sf, masked_m=(count - lo).clamp(min=0).to(torch.int32))
        else:
            run(part[0], q[0], sf[0], m_indices=m[lo:hi], **more)
        return [q, sf, *more.values()]

    whole = call(0, rows)
    step = rows // 4
    parts = [call(lo, lo + step) for lo in range(0, rows, step)]
    row_axis = [1, 2, 0, 1]
    for n, got in enumerate(whole):
        assert torch.equal(got, torch.cat([p[n] for p in parts], row_axis[n])), n


# ------------------------------------------------------------------ combine --

@pytest.mark.parametrize("groups,m_max,cols", [(1, 4, 128), (4, 37, 1152), (32, 16, 7168)])
def test_combine_of_the_masked_layout(groups, m_max, cols):
    dg = require_gpu()
    rng = np.random.default_rng(groups + cols)
    tokens, topk = 33, 5
    d = synth.bf16_normal((groups * m_max, cols), 130)
    rows = rng.integers(-1, groups * m_max + 2, (tokens, topk)).astype(np.int32)
    w = rng.random((tokens, topk)).astype(np.float32)
    y = torch.empty(tokens, cols, dtype=torch.bfloat16, device="cuda")
    td, tr, tw = dev(d).view(groups, m_max, cols), torch.as_tensor(rows, device="cuda"), torch.as_tensor(w, device="cuda")
    dg.dg_moe_combine(td, tr, y, weights=tw)
    ref, size = moe.combine(bf16_to_f64(d), rows, w)
    assert np.all(np.abs(bf16_to_f64(host(y)) - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -22 * topk * size)
    if groups > 1:
        with pytest.raises(ValueError, match="contiguous"):
            dg.dg_moe_combine(td.transpose(0, 1), tr, y, weights=tw)


# ------------------------------------------------------- forward, both layouts --

@pytest.mark.parametrize("ue8m0", [False, True])
@pytest.mark.parametrize("layout", ["masked", "contiguous"])
@pytest.mark.parametrize("tokens,hidden,inter,experts,topk,first,local", [
    (1, 256, 128, 8, 8, 0, 8), (128, 512, 384, 32, 4, 8, 16), (300, 384, 256, 16, 2, 0, 16)])
def test_forward_against_float32(layout, ue8m0, tokens, hidden, inter, experts, topk, first, local):
    """route, plan, dispatch, grouped GEMM, gated unit, grouped GEMM, combine for the
    experts [first, first + local) of one device.  Four quantisations of 2.6 % each
    (3 mantissa bits), two of them through the unit: bound 10 %."""
    dg = require_gpu()
    g = torch.Generator(device="cuda").manual_seed(tokens)
    normal = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    x, logits = normal(tokens, hidden).bfloat16(), 1.5 * normal(tokens, experts)
    w1 = (normal(local, 2 * inter, hidden) / hidden ** 0.5).bfloat16()
    w2 = (normal(local, hidden, inter) / inter ** 0.5).bfloat16()

    def weights_of(w):
        n, k = w.shape[1:]
        q = torch.empty(w.shape, dtype=torch.uint8, device="cuda")
        if ue8m0:
            sf = torch.empty(local, k // 128, dg.dg_get_ue8m0_sfb_leading_dim(n), dtype=torch.uint8, device="cuda")
            dg.dg_quant_128x128_ue8m0(w, q, sf)
        else:
            sf = torch.empty(local, (n + 127) // 128, k // 128, device="cuda")
            dg.dg_quant_128x128(w, q, sf)
        return q, sf

    b1, b2 = weights_of(w1), weights_of(w2)
    i32 = lambda *s: torch.empty(s, dtype=torch.int32, device="cuda")  # noqa: E731
    bf = lambda *s: torch.empty(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    ids, weights, rows, y = i32(tokens, topk), torch.empty(tokens, topk, device="cuda"), i32(tokens, topk), bf(tokens, hidden)
    dg.dg_moe_route(logits, ids, weights, score="sigmoid", scale=2.5)
    ws = torch.empty(max(16, dg.dg_get_moe_plan_workspace_size(tokens, topk, local)), dtype=torch.uint8, device="cuda")
    masked = layout == "masked"
    m = (tokens + 3) // 4 * 4 if masked else (tokens * topk + 127 * local + 127) // 128 * 128
    shape, sf_shape = ((local, m), (local,)) if masked else ((m,), ())
    src = i32(local * m if masked else m)
    if masked:
        use = dict(masked_m=i32(local))
        dg.dg_moe_plan_masked(ids, rows, src, use["masked_m"], first_expert=first, workspace=ws)
    else:
        use = dict(m_indices=i32(m))
        dg.dg_moe_plan_contiguous(ids, rows, src, use["m_indices"], i32(local + 1), first_expert=first, workspace=ws)
    new_sf = lambda cols: torch.empty((*sf_shape, cols // 128, m), dtype=torch.uint8 if ue8m0 else torch.float32, device="cuda")  # noqa: E731
    a, asf, act, actsf = _u8(*shape, hidden), new_sf(hidden), _u8(*shape, inter), new_sf(inter)
    h, d = bf(*shape, 2 * inter), bf(*shape, hidden)
    gemm = {(True, False): dg.dg_grouped_masked, (True, True): dg.dg_grouped_masked_ue8m0,
            (False, False): dg.dg_grouped_contiguous, (False, True): dg.dg_grouped_contiguous_ue8m0}[masked, ue8m0]
    gws = torch.zeros(max(16, dg.dg_get_workspace_size(m, 2 * inter, hidden, local), dg.dg_get_workspace_size(m, hidden, inter, local)),
                      dtype=torch.uint8, device="cuda")
    index = next(iter(use.values()))
    (dg.dg_moe_dispatch_ue8m0 if ue8m0 else dg.dg_moe_dispatch)(x, src, a, asf, topk=topk)
    gemm(a, asf, *b1, h, index, workspace=gws)
    (dg.dg_swiglu_quant_ue8m0 if ue8m0 else dg.dg_swiglu_quant)(h, act, actsf, **use)
    gemm(act, actsf, *b2, d, index, workspace=gws)
    dg.dg_moe_combine(d, rows, y, weights=weights)

    want = torch.zeros(tokens, hidden, device="cuda")
    for e in range(local):
        t, j = (ids == first + e).nonzero(as_tuple=True)
        gate, up = (x[t].float() @ w1[e].float().t()).chunk(2, dim=1)
        want.index_add_(0, t, weights[t, j, None] * ((torch.nn.functional.silu(gate) * up) @ w2[e].float().t()))
    assert float((y.float() - want).norm() / want.norm()) < 0.10
    gone = ((ids < first) | (ids >= first + local)).all(1)
    assert not y[gone].any()
