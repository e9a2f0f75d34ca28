"""GPU 8-bit activation checkpoints (dg_swiglu_quant*, dg_swiglu_bwd,
dg_requant_t) against oracle/moe.py and the oracle's quantisers.

The checkpoint equals the activation quantiser's output bit for bit.  Codes of
computed values must be a nearest e4m3 number of v / s for a v / s within
2^-18 of the oracle's (float32 sigmoids of moderate gates carry about 2^-21),
scales within 2^-20 of the oracle's; UE8M0 exponents equal the oracle's unless
amax / 448 lies within 2^-20 of a power of two.
"""

import numpy as np
import pytest
import torch

import synth
from oracle import e4m3, moe, quant
from tests.gpu_util import bf16_to_f64, dev, host, require_gpu
from tests.test_gpu_moe_exchange import FILL, check_codes, check_transposed

pytestmark = pytest.mark.gpu


def _u8(*shape):
    return torch.full(shape, FILL, dtype=torch.uint8, device="cuda")


def _f32(*shape):
    return torch.full(shape, -3.0, device="cuda")


def make_h(rows, inter, seed, scale=1.5):
    h = synth.bf16_normal((rows, 2 * inter), seed, scale)
    h[0, :128] = 0                  # a gate tile of zeros: an all-zero tile of the unit's output
    if rows > 1:
        h[1, :8] = 0xC2C8           # gates of -100: silu underflows to a tiny number
        h[1, 8:16] = 0x42C8         # and of 100
    return h


def segments(rng, m_total, empty_tail):
    m = np.full(m_total, -1, dtype=np.int32)
    for b in range(m_total // 128 - empty_tail):
        m[b * 128:b * 128 + rng.integers(1, 129)] = b % 3
    return m


def _rows_check(q, sf, v, live):
    q, sf = host(q), host(sf)
    rows = len(v)
    assert np.all(q[~live] == FILL) and np.all(sf[:, :rows][:, ~live] == -3.0) and np.all(sf[:, rows:] == -3.0)
    check_codes(q[live], np.repeat(sf[:, :rows].T, 128, axis=1)[live], v[live],
                np.repeat(moe.row_scales(v).T, 128, axis=1)[live], slice(None), "rows")


@pytest.mark.parametrize("ckpt", [False, True])
@pytest.mark.parametrize("rows,inter,pad,ld,mask", [
    (1, 128, 0, 4, False), (37, 256, 8, 44, False), (256, 1152, 0, 256, True), (640, 2048, 16, 644, True), (5, 4096, 0, 8, False)])
def test_swiglu_quant_contiguous(ckpt, rows, inter, pad, ld, mask):
    dg = require_gpu()
    rng = np.random.default_rng(rows + inter)
    h = make_h(rows, inter, 91)
    m = segments(rng, rows, 1) if mask else None
    live = m >= 0 if mask else np.ones(rows, dtype=bool)
    h[~live] = 0x7FC0
    q, sf = _u8(rows, inter), _f32(inter // 128, ld)
    hq, hsf = (_u8(rows, 2 * inter), _f32(inter // 64, ld)) if ckpt else (None, None)
    th = dev(np.pad(h, ((0, 0), (0, pad))))[:, :2 * inter]
    dg.dg_swiglu_quant(th, q, sf, m_indices=None if m is None else torch.as_tensor(m, device="cuda"), hq=hq, hsf=hsf)
    v = np.where(live[:, None], moe.swiglu(bf16_to_f64(np.where(live[:, None], h, 0))), 0.0)
    _rows_check(q, sf, v, live)
    if ckpt:
        ref_q, ref_sf = quant.quant_1x128(np.where(live[:, None], h, 0).astype(np.uint16))
        got_q, got_sf = host(hq), host(hsf)
        assert np.array_equal(got_q[live], ref_q[live]) and np.all(got_q[~live] == FILL)
        assert np.array_equal(got_sf[:, :rows][:, live], ref_sf[:, :rows][:, live])
        assert np.all(got_sf[:, :rows][:, ~live] == -3.0) and np.all(got_sf[:, rows:] == -3.0)


@pytest.mark.parametrize("ue", [False, True])
@pytest.mark.parametrize("groups,m_max,inter,ld", [(1, 1, 128, 4), (3, 17, 256, 20), (32, 128, 2048, 128), (5, 300, 384, 304)])
def test_swiglu_quant_masked(ue, groups, m_max, inter, ld):
    dg = require_gpu()
    rng = np.random.default_rng(groups + inter)
    h = make_h(groups * m_max, inter, 92)
    count = rng.integers(0, m_max + 1, groups).astype(np.int32)
    count[0], count[-1] = m_max + 5, (0 if groups > 1 else m_max)  # past the end: clamped; none
    live = (np.arange(m_max)[None, :] < count[:, None]).reshape(-1)
    h[~live] = 0x7FC0
    q = _u8(groups, m_max, inter)
    sf = torch.full((groups, inter // 128, ld), 0x5A, dtype=torch.uint8, device="cuda") if ue else _f32(groups, inter // 128, ld)
    (dg.dg_swiglu_quant_ue8m0 if ue else dg.dg_swiglu_quant)(
        dev(h).view(groups, m_max, 2 * inter), q, sf, masked_m=torch.as_tensor(count, device="cuda"))
    v = np.where(live[:, None], moe.swiglu(bf16_to_f64(np.where(live[:, None], h, 0))), 0.0)
    for g in range(groups):
        part = slice(g * m_max, (g + 1) * m_max)
        if not ue:
            _rows_check(q[g], sf[g], v[part], live[part])
            continue
        s = host(sf[g])
        mine = live[part]
        assert np.all(s[:, :m_max][:, ~mine] == 0x5A) and np.all(s[:, m_max:] == 0x5A)
        if not mine.any():
            continue
        amax = np.abs(v[part][mine]).reshape(int(mine.sum()), -1, 128).max(2).T
        got = s[:, :m_max][:, mine].astype(np.int64)
        with np.errstate(divide="ignore"):
            exact = np.log2(amax / 448.0)
        e = np.where(amax > 0, np.clip(np.ceil(exact), -127, 127) + 127, 0).astype(np.int64)
        near = np.abs(exact - np.round(exact)) < 2.0 ** -20
        assert np.all((got == e) | (near & (np.abs(got - e) <= 1)))
        t = v[part][mine] / np.repeat(np.ldexp(1.0, (got - 127)).T, 128, axis=1)
        off = np.abs(e4m3.decode(host(q[g])[mine]).astype(np.float64) - t)
        assert np.all(off <= moe.half_step(np.abs(t) * (1 + 2.0 ** -18)) + 2.0 ** -18 * np.abs(t))


@pytest.mark.parametrize("with_act", [True, False])
@pytest.mark.parametrize("m_total,inter,mask,tail,pad", [
    (128, 128, False, 0, 0), (128, 256, True, 0, 8), (640, 384, True, 2, 0), (384, 2048, True, 1, 0)])
def test_swiglu_bwd(with_act, m_total, inter, mask, tail, pad):
    dg = require_gpu()
    rng = np.random.default_rng(m_total + inter)
    m = segments(rng, m_total, tail) if mask else np.zeros(m_total, dtype=np.int32)
    live = m >= 0
    hq, hsf = quant.quant_1x128(make_h(m_total, inter, 93))
    da = synth.bf16_normal((m_total, inter), 94)
    da[2 % m_total, :128] = 0
    hq[~live], da[~live] = 0x7F, 0x7FC0  # NaN where no row is in use
    hsf = np.where(np.concatenate([live, np.zeros(hsf.shape[1] - m_total, dtype=bool)])[None], hsf, np.nan).astype(np.float32)
    out = dict(dq=_u8(m_total, 2 * inter), dsf=_f32(inter // 64, m_total + 4), dqt=_u8(2 * inter, m_total),
               dsft=_f32(m_total // 128, 2 * inter + 4))
    if with_act:
        out |= dict(aqt=_u8(inter, m_total), asft=_f32(m_total // 128, inter + 12))
    tda = dev(np.pad(da, ((0, 0), (0, pad))))[:, :inter]
    dg.dg_swiglu_bwd(dev(hq), dev(hsf), tda, torch.as_tensor(m, device="cuda") if mask else None, **out)
    h = np.where(live[:, None], moe.dequant_rows(np.where(live[:, None], hq, 0), np.nan_to_num(hsf)), 0.0)
    dh = np.where(live[:, None], moe.swiglu_bwd(h, bf16_to_f64(np.where(live[:, None], da, 0))), 0.0)
    _rows_check(out["dq"], out["dsf"], dh, live)
    check_transposed(host(out["dqt"]), host(out["dsft"]), dh, live, 2 * inter)
    if with_act:
        check_transposed(host(out["aqt"]), host(out["asft"]), moe.swiglu(h), live, inter)


@pytest.mark.parametrize("rows,cols,mask,tail", [(128, 128, False, 0), (256, 384, True, 0), (640, 1152, True, 2), (384, 7168, False, 0)])
def test_requant_t(rows, cols, mask, tail):
    dg = require_gpu()
    rng = np.random.default_rng(rows + cols)
    m = segments(rng, rows, tail) if mask else np.zeros(rows, dtype=np.int32)
    live = m >= 0
    q, sf = quant.quant_1x128(make_h(rows, cols // 2, 95, 3.0))
    q[~live] = 0x7F
    sf[:, :rows][:, ~live] = np.nan
    qt, sft = _u8(cols, rows), _f32(rows // 128, cols + 4)
    dg.dg_requant_t(dev(q), dev(sf), torch.as_tensor(m, device="cuda") if mask else None, qt, sft)
    v = np.where(live[:, None], moe.dequant_rows(np.where(live[:, None], q, 0), np.nan_to_num(sf)), 0.0)
    check_transposed(host(qt), host(sft), v, live, cols)


def test_tiny_values_keep_finite_scales():
    """Tiles whose largest value is a float32 subnormal: scale 2^-126, finite codes."""
    dg = require_gpu()
    q = np.full((128, 128), 0x38, dtype=np.uint8)  # 1.0
    sf = np.full((1, 128), 2.0 ** -140, dtype=np.float32)
    sf[0, 5] = 0.0
    qt, sft = _u8(128, 128), _f32(1, 128)
    dg.dg_requant_t(dev(q), dev(sf), None, qt, sft)
    assert np.all(host(sft) == np.float32(2.0 ** -126))
    got = e4m3.decode(host(qt)).astype(np.float64)
    assert np.all(got == 0)  # 2^-140 / 2^-126 is far below the smallest code


def test_large_offsets():
    """A checkpoint of more than 2^32 codes: the last blocks are addressed with 64 bits."""
    dg = require_gpu()
    rows, cols = 614400, 7168
    m = torch.full((rows,), -1, dtype=torch.int32, device="cuda")
    m[rows - 256:rows - 3] = 0
    q = torch.full((rows, cols), 0x7F, dtype=torch.uint8, device="cuda")
    sf = torch.full((cols // 128, rows), float("nan"), device="cuda")
    tail, tail_sf = quant.quant_1x128(synth.bf16_normal((256, cols), 96))
    q[rows - 256:], sf[:, rows - 256:] = dev(tail), dev(tail_sf)
    qt, sft = torch.zeros((cols, rows), dtype=torch.uint8, device="cuda"), _f32(rows // 128, cols)
    dg.dg_requant_t(q, sf, m, qt, sft)
    live = host(m[rows - 256:]) >= 0
    v = np.where(live[:, None], moe.dequant_rows(tail, tail_sf), 0.0)
    check_transposed(host(qt[:, rows - 256:].contiguous()), host(sft[-2:]), v, live, cols)
    assert int(qt[:, :rows - 256].ne(0).sum()) == 0 and bool((sft[:-2] == -3.0).all())
