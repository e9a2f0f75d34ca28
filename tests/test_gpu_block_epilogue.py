"""GPU GEMM with an epilogue (dg_fp8_gemm_nt_epilogue, dg_fp8_gemm_nt_ue8m0_epilogue)
and its gradient (dg_epilogue_bwd) against oracle/gemm.py and oracle/block.py.

The sum of random operands is held to the rule of every GEMM comparison
(tests/tolerance.py): 1e-2 of the sums' root mean square before the rounding.  The
matrix core does not keep all bits of a slice's products: next to one of exponents
ea + eb = E it drops what others have below 2^(E - 13) (products of 1.0 and of 16
beside +-448 and +-16 that cancel), so a slice of 128 products can lose up to
128 * 2^-13 = 2^-6 of its largest one, which is about a tenth of a slice's root mean
square times 2^-6 * 8: the rule's 1e-2.  Where the products are small integers nothing
is dropped (|sum| and every product are multiples of 1 below 2^13), the sum is exact,
and the epilogue alone is left: LOST_EXACT.  Activations have slopes of at most 1.13
and lose 2^-20 of themselves; d and z are rounded once (2^-8).  Without an epilogue's
terms the result is that of dg_fp8_gemm_nt bit for bit, and the quantised copy is the
quantiser's of d.
"""

import numpy as np
import pytest
import torch

from oracle import block, e4m3, gemm, moe, quant, ue8m0
from synth import bf16_normal
from tests.block_util import (FILL, SENTINEL, UNWRITTEN, check_codes, check_f32, check_row_codes, check_scales, code_buffers,
                              empty_rows, f32, padded, pads_kept, workspace)
from tests import tolerance
from tests.gpu_util import bf16_to_f64, dev, host, require_gpu

pytestmark = pytest.mark.gpu

ACTS = ["none", "relu", "silu", "gelu_tanh"]

# Of the terms' magnitudes, where the sum is exact: a bias, an activation (2^-20) and a residual, each rounded in
# float32.
LOST_EXACT = 2.0 ** -19


class Operands:
    def __init__(self, dg, m, n, k, ue, seed=70):
        xa, xb = bf16_normal((m, k), seed), bf16_normal((n, k), seed + 1, k ** -0.5)
        if ue:
            self.a, self.sfa = ue8m0.quant_1x128_ue8m0(xa)
            self.b, self.sfb = ue8m0.quant_128x128_ue8m0(xb)
            fa, fb = ue8m0.sfa_as_fp32(self.sfa), ue8m0.sfb_as_fp32(self.sfb, n)
        else:
            self.a, self.sfa = quant.quant_1x128(xa)
            self.b, self.sfb = quant.quant_128x128(xb)
            fa, fb = self.sfa, self.sfb
        self.z = gemm.gemm_nt_ref(self.a, fa, self.b, fb)
        self.off = tolerance.ABS_RMS * np.sqrt((self.z ** 2).mean())  # what a sum may be off by
        self.dev = [dev(v) for v in (self.a, self.sfa, self.b, self.sfb)]
        size = dg.dg_get_workspace_size(m, n, k)
        self.ws = torch.zeros(size, dtype=torch.uint8, device="cuda") if size else None
        self.gemm = dg.dg_fp8_gemm_nt_ue8m0_epilogue if ue else dg.dg_fp8_gemm_nt_epilogue
        self.plain = dg.dg_fp8_gemm_nt_ue8m0 if ue else dg.dg_fp8_gemm_nt


def check_d(got, want, off, what):
    """bf16 results of values that may be off by `off`."""
    got = bf16_to_f64(host(got))
    bad = ~(np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + off + 2.0 ** -134)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size}, first at {np.argwhere(bad)[0]}: {got[bad][0]} for {want[bad][0]}"


def run(ops, m, n, act, bias, res, pre, ld, seed=80):
    rng = np.random.default_rng(seed)
    b = rng.standard_normal(n).astype(np.float32) if bias else None
    r = bf16_normal((m, n), seed) if res else None
    d, z = empty_rows(m, n, ld - n), empty_rows(m, n, ld - n) if pre else None
    ops.gemm(*ops.dev, d, bias=f32(b), act=act, residual=None if r is None else padded(r, ld - n), pre=z, workspace=ops.ws)
    want = ops.z.copy()
    if bias:
        want = want + b.astype(np.float64)
    if pre:
        check_d(z, want, ops.off, "z")
        assert pads_kept(z)
    want = block.act(want, act)
    off = 1.13 * ops.off + 2.0 ** -20 * np.abs(want)
    if res:
        want = want + bf16_to_f64(r)
    check_d(d, want, off + 2.0 ** -24 * np.abs(want), "d")
    assert pads_kept(d)
    return d, z


SHAPES = [(1, 16, 128), (1, 7168, 2048), (3, 5, 256), (33, 83, 128), (64, 2109, 1024), (128, 200, 384), (130, 1001, 512),
          (257, 386, 7168), (300, 4099, 256), (2049, 514, 128)]


@pytest.mark.parametrize("m,n,k", SHAPES)
@pytest.mark.parametrize("ue", [False, True])
def test_epilogue(m, n, k, ue):
    dg = require_gpu()
    ops = Operands(dg, m, n, k, ue)
    ld = (n + 7) // 8 * 8 + 8
    for i, act in enumerate(ACTS):
        run(ops, m, n, act, bias=i != 1, res=i % 2 == 0, pre=i > 1, ld=ld)
    # Nothing to do after the sum: the plain GEMM, bit for bit.
    d, want = empty_rows(m, n, ld - n), empty_rows(m, n, ld - n)
    ops.gemm(*ops.dev, d, workspace=ops.ws)
    ops.plain(*ops.dev, want, workspace=ops.ws)
    assert torch.equal(d, want)


class ExactOperands(Operands):
    """Operands of small integers with scales of 1: every sum is an exact integer."""

    def __init__(self, dg, m, n, k, ue):
        super().__init__(dg, m, n, k, ue)
        rng = np.random.default_rng(m + n + k)
        va, vb = rng.integers(-2, 3, (m, k)).astype(np.float64), (rng.integers(-2, 3, (n, k)) * (rng.random((n, k)) < 0.2)).astype(np.float64)
        self.z, self.off = va @ vb.T, 0.0
        one = lambda sf: np.full(sf.shape, 127, dtype=np.uint8) if ue else np.ones(sf.shape, dtype=np.float32)
        self.dev = [dev(e4m3.encode_rne(va)), dev(one(self.sfa)), dev(e4m3.encode_rne(vb)), dev(one(self.sfb))]


@pytest.mark.parametrize("m,n,k", SHAPES)
@pytest.mark.parametrize("ue", [False, True])
@pytest.mark.parametrize("act", ACTS)
def test_epilogue_of_exact_sums(m, n, k, ue, act):
    dg = require_gpu()
    ops = ExactOperands(dg, m, n, k, ue)
    d, z, plain = (empty_rows(m, n, (-n) % 8) for _ in range(3))
    ops.plain(*ops.dev, plain, workspace=ops.ws)
    check_d(plain, ops.z, 0.0, "sum")
    rng = np.random.default_rng(4)
    bias, res = (rng.integers(-64, 65, n) / 16).astype(np.float32), bf16_normal((m, n), 5, 4.0)
    ops.gemm(*ops.dev, d, bias=f32(bias), act=act, residual=padded(res, (-n) % 8), pre=z, workspace=ops.ws)
    want = ops.z + bias
    check_d(z, want, 0.0, "z")
    out = block.act(want, act)
    check_d(d, out + bf16_to_f64(res), LOST_EXACT * (np.abs(want) + np.abs(bf16_to_f64(res))), "d")


@pytest.mark.parametrize("variant", [0, 4, 5, 6, 11])
@pytest.mark.parametrize("division", [0, 1, 3])
@pytest.mark.parametrize("ue", [False, True])
def test_every_tile_and_work_division(variant, division, ue, monkeypatch):
    dg = require_gpu()
    if ue and variant == 11:
        pytest.skip("the 256 x 160 tile has no UE8M0 form")
    m, n, k = 150, 391, 1536
    monkeypatch.setenv("DG_FORCE_CONFIG", f"{variant}:{division}:{division % 2}")
    ops = Operands(dg, m, n, k, ue)
    d, z = run(ops, m, n, "silu", True, True, True, 400)
    # Partial sums are added in a fixed order, and the epilogue follows once.
    again, z2 = run(ops, m, n, "silu", True, True, True, 400)
    assert torch.equal(d, again) and torch.equal(z, z2)


def test_tiles_without_an_epilogue_are_refused(monkeypatch):
    dg = require_gpu()
    ops = Operands(dg, 150, 391, 256, False)
    for variant in (1, 2, 3, 7, 8, 9, 10):
        monkeypatch.setenv("DG_FORCE_CONFIG", f"{variant}:0")
        d = empty_rows(150, 391, 1)
        with pytest.raises(dg.DGError, match="epilogue"):
            ops.gemm(*ops.dev, d, workspace=ops.ws)
        assert bool((d == SENTINEL).all())


@pytest.mark.parametrize("m,n,k", [(1, 128, 128), (64, 4096, 7168), (150, 384, 1536), (300, 2048, 256)])
@pytest.mark.parametrize("ue", [False, True])
def test_quantised_copy(m, n, k, ue):
    dg = require_gpu()
    ops = Operands(dg, m, n, k, ue)
    rng = np.random.default_rng(1)
    bias = f32(rng.standard_normal(n))
    d, z = empty_rows(m, n), empty_rows(m, n)
    ld = (m + 3) // 4 * 4 + 4
    dq, dsf = code_buffers(m, n, ld, ue)
    ops.gemm(*ops.dev, d, bias=bias, act="gelu_tanh", pre=z, dq=dq, dsf=dsf, workspace=ops.ws)
    want = ops.z + host(bias).astype(np.float64)
    check_d(z, want, ops.off, "z")
    check_d(d, block.act(want, "gelu_tanh"), 1.13 * ops.off + 2.0 ** -20 * np.abs(want), "d")
    q, sf = (ue8m0.quant_1x128_ue8m0 if ue else quant.quant_1x128)(host(d), ld)
    assert np.array_equal(host(dq), q) and np.array_equal(host(dsf), sf)


def test_empty_sum_keeps_its_epilogue():
    dg = require_gpu()
    m, n = 70, 130
    rng = np.random.default_rng(2)
    bias, res = rng.standard_normal(n).astype(np.float32), bf16_normal((m, n), 3)
    d = empty_rows(m, n, 6)
    a, b = torch.zeros(m, 0, dtype=torch.uint8, device="cuda"), torch.zeros(n, 0, dtype=torch.uint8, device="cuda")
    dg.dg_fp8_gemm_nt_epilogue(a, torch.zeros(0, 72, device="cuda"), b, torch.zeros(2, 0, device="cuda"), d, bias=f32(bias),
                               act="silu", residual=padded(res, 6))
    want = block.act(np.broadcast_to(bias, (m, n)), "silu") + bf16_to_f64(res)
    check_d(d, want, LOST_EXACT * (np.abs(bias) + np.abs(bf16_to_f64(res))), "d")
    empty = torch.zeros(0, n + 6, dtype=torch.bfloat16, device="cuda")[:, :n]
    dg.dg_fp8_gemm_nt_epilogue(a[:0], torch.zeros(0, 4, device="cuda"), b, torch.zeros(2, 0, device="cuda"), empty)


def test_large_values_meet_the_activations():
    """Sums of +-2^100 and +-300: activations saturate, nothing overflows on the way."""
    dg = require_gpu()
    m, n, k = 4, 8, 128
    a, b = torch.zeros(m, k, dtype=torch.uint8, device="cuda"), torch.zeros(n, k, dtype=torch.uint8, device="cuda")
    bias = torch.tensor([2.0 ** 100, -2.0 ** 100, 300.0, -300.0, 20.0, -20.0, 0.0, -0.0], device="cuda")
    for act in ACTS:
        d = torch.empty(m, n, dtype=torch.bfloat16, device="cuda")
        dg.dg_fp8_gemm_nt_epilogue(a, torch.zeros(1, 4, device="cuda"), b, torch.zeros(1, 1, device="cuda"), d, bias=bias, act=act)
        want = block.act(bias.double().cpu().numpy(), act)
        got = d.double().cpu().numpy()
        assert np.all(np.abs(got - want) <= (2.0 ** -8 + 2.0 ** -20) * np.abs(want) + 1e-38), act


def test_epilogue_in_a_graph_with_split_sums():
    dg = require_gpu()
    m, n, k = 64, 4096, 7168
    ops = Operands(dg, m, n, k, False)
    assert ops.ws is not None
    bias = torch.zeros(n, device="cuda")
    d, dq, dsf = torch.empty(m, n, dtype=torch.bfloat16, device="cuda"), *code_buffers(m, n, m)
    dd, gq, gsf = torch.empty_like(d), *code_buffers(m, n, m)
    gqt, gsft = torch.zeros(n, 128, dtype=torch.uint8, device="cuda"), torch.zeros(1, n, device="cuda")
    z, db = torch.empty_like(d), torch.zeros(n, device="cuda")

    def step():
        ops.gemm(*ops.dev, d, bias=bias, act="silu", pre=z, workspace=ops.ws)
        dd.copy_(d)
        dg.dg_epilogue_bwd(dd, gq, gsf, pre=z, act="silu", dqt=gqt, dsft=gsft, dbias=db)
        return [v.clone() for v in (d, z, gq, gsf, gqt, gsft, db)]

    sets = [torch.randn(n, device="cuda") for _ in range(3)]
    want = []
    for v in sets:
        bias.copy_(v)
        want.append(step())
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for x, y in zip(step(), want[2]):
            assert torch.equal(x, y)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for i in (0, 2, 1, 0):
        bias.copy_(sets[i])
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(got, want[i]):
            assert torch.equal(x, y)


# -------------------------------------------------------------- gradient --

@pytest.mark.parametrize("rows,cols,pad", [(1, 128, 0), (3, 384, 8), (64, 128, 0), (127, 256, 16), (128, 1152, 0), (129, 512, 0),
                                           (1001, 2048, 8), (2600, 640, 0)])
@pytest.mark.parametrize("act", ACTS)
def test_epilogue_bwd(rows, cols, pad, act):
    dg = require_gpu()
    dd, z = bf16_normal((rows, cols), 90), bf16_normal((rows, cols), 91, 2.0)
    z[0, :8] = [0, 0x8000, 0x42C8, 0xC2C8, 0x7149, 0xF149, 0xBFA4, 0xBF40]  # 0, -0, +-100, +-1e30, -1.28, -0.75
    dd[:, 128:256] = 0  # tiles of zeros, where there is a second one
    ld = (rows + 3) // 4 * 4 + 4
    dq, dsf = code_buffers(rows, cols, ld)
    tiles = -(-rows // 128)
    dqt = torch.full((cols, tiles * 128), FILL, dtype=torch.uint8, device="cuda")
    dsft = torch.full((tiles, cols + 4), UNWRITTEN, device="cuda")
    db = torch.full((cols,), float("nan"), device="cuda")
    ws = workspace(dg.dg_get_epilogue_bwd_workspace_size(rows, cols))
    tdd, tz = padded(dd, pad), None if act == "none" else padded(z, pad)
    dg.dg_epilogue_bwd(tdd, dq, dsf, pre=tz, act=act, dqt=dqt, dsft=dsft, dbias=db, workspace=ws)
    g = bf16_to_f64(dd)
    v = g * block.act_slope(bf16_to_f64(z), act)
    # A slope is a sum of two terms, sigmoid and z sigmoid', of at most 1 and 1.13 in all; the product loses 2^-20.
    mag = np.abs(g) * (1.0 if act != "none" else 0.0)
    check_row_codes(dq, dsf, v, mag, False, "rows")
    wide, wmag = np.zeros((tiles * 128, cols)), np.zeros((tiles * 128, cols))
    wide[:rows], wmag[:rows] = v, mag
    q, sf = host(dqt), host(dsft)
    assert np.all(sf[:, cols:] == UNWRITTEN) and np.all(q[:, rows:] & 0x7F == 0)
    by = lambda a: np.abs(a).reshape(tiles, 128, cols).max(1)
    check_scales(sf[:, :cols], by(wide), by(wmag), "columns")
    check_codes(q, np.repeat(sf[:, :cols].T, 128, axis=1), wide.T, wmag.T, "columns")
    check_f32(db, v.sum(0), np.abs(v).sum(0) + mag.sum(0), "dbias")
    # Parts of it, and twice the same.
    dq2, dsf2 = code_buffers(rows, cols, ld)
    dg.dg_epilogue_bwd(tdd, dq2, dsf2, pre=tz, act=act)
    assert torch.equal(dq2, dq) and torch.equal(dsf2, dsf)
    db2 = torch.zeros(cols, device="cuda")
    dg.dg_epilogue_bwd(tdd, dq2, dsf2, pre=tz, act=act, dbias=db2, workspace=workspace(ws.numel(), 0xFF))
    assert torch.equal(db2, db)


def test_epilogue_bwd_of_no_rows():
    dg = require_gpu()
    db = torch.full((256,), 5.0, device="cuda")
    dg.dg_epilogue_bwd(torch.zeros(0, 256, dtype=torch.bfloat16, device="cuda"), torch.zeros(0, 256, dtype=torch.uint8, device="cuda"),
                       torch.zeros(2, 4, device="cuda"), dbias=db)
    assert not db.any()


def test_gradient_products_take_the_codes():
    """dz's codes as the operands that they are: input gradient by rows, weight gradient transposed, against the
    products of the values that the codes stand for."""
    dg = require_gpu()
    rows, cols, k = 200, 384, 256
    dd, z = bf16_normal((rows, cols), 95), bf16_normal((rows, cols), 96, 2.0)
    wide = 256
    dq, dsf = torch.zeros(rows, cols, dtype=torch.uint8, device="cuda"), torch.zeros(cols // 128, rows, device="cuda")
    dqt, dsft = torch.zeros(cols, wide, dtype=torch.uint8, device="cuda"), torch.zeros(wide // 128, cols, device="cuda")
    dg.dg_epilogue_bwd(dev(dd), dq, dsf, pre=dev(z), act="gelu_tanh", dqt=dqt, dsft=dsft)
    wq, wsf = quant.quant_128x128(bf16_normal((k, cols), 97))  # the weight transposed: [in][out]
    dx = torch.zeros(rows, k, dtype=torch.bfloat16, device="cuda")
    dg.dg_fp8_gemm_nt(dq, dsf, dev(wq), dev(wsf), dx)
    want = gemm.gemm_nt_ref(host(dq), host(dsf), wq, wsf)
    tolerance.check(bf16_to_f64(host(dx)), want, "dx")
    x = bf16_normal((k, wide), 98)  # the input transposed; columns past the rows hold whatever padding holds
    xq, sfx = quant.quant_1x128(x)
    dw = torch.zeros(1, cols, k, dtype=torch.bfloat16, device="cuda")
    ends = torch.tensor([0, wide], dtype=torch.int32, device="cuda")
    dg.dg_k_grouped_nt(dqt, dsft, dev(xq), dev(sfx), dw, ends)
    zt = moe.dequant_rows(host(dqt), host(dsft))
    xt = moe.dequant_rows(xq, sfx)
    tolerance.check(bf16_to_f64(host(dw[0])), zt @ xt.T, "dw")
    # The codes stand for dz: within half a step of e4m3 (2^-4) of every value, and of the tile's smallest steps.
    v = bf16_to_f64(dd) * block.act_slope(bf16_to_f64(z), "gelu_tanh")
    top = np.repeat(np.abs(np.pad(v, ((0, wide - rows), (0, 0)))).reshape(2, 128, cols).max(1), 128, axis=0)[:rows]
    assert np.all(np.abs(zt.T[:rows] - v) <= 2.0 ** -4 * np.abs(v) * 1.001 + 2.0 ** -10 * top / 448.0 * 1.001 + 1e-6 * top)
