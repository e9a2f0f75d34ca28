"""GPU norms fused with gate and residual (dg_block_norm*, dg_block_norm_bwd)
against oracle/block.py; tolerances in tests/block_util.py."""

import numpy as np
import pytest
import torch

import synth
from oracle import block
from tests.block_util import (check_exponents, check_f32, check_row_codes, check_rows, code_buffers, empty_rows, f32, padded,
                              pads_kept, workspace)
from tests.gpu_util import bf16_to_f64, dev, host, require_gpu

pytestmark = pytest.mark.gpu


def rows_of(tokens, cols, seed):
    """bf16 bits of rows of very different sizes, one of zeros and one with a mean far from zero among them."""
    rng = np.random.default_rng(seed)
    v = synth.bf16_normal((tokens, cols), seed)
    scale = np.exp2(rng.integers(-12, 13, (tokens, 1)))
    f = (bf16_to_f64(v) * scale).astype(np.float32)
    if tokens > 2:
        f[1] = 0.0
        f[2] += 40.0 * scale[2]
    return (f.view(np.uint32) >> 16).astype(np.uint16)  # cut: any bf16 will do


def parameters(tokens, cols, seed, gate, bias, post):
    rng = np.random.default_rng(seed)
    draw = lambda *s: rng.standard_normal(s).astype(np.float32)
    out = {"weight": 1 + 0.2 * draw(cols)}
    if bias:
        out["bias"] = draw(cols)
    if post:
        out["post_weight"] = 1 + 0.2 * draw(cols)
    if gate:
        out["gate"] = draw(cols) if gate == "column" else draw(tokens, 1)
    return out


SIZES = [(1, 8, 0), (3, 40, 8), (100, 128, 0), (37, 136, 8), (45, 256, 0), (5, 512, 0), (9, 1000, 16), (130, 1024, 0), (6, 1536, 0), (33, 2048, 8), (4, 3584, 0),
         (7, 4104, 8), (5, 6144, 0), (300, 7168, 0), (3, 8192, 0), (2, 8200, 0), (3, 16384, 8)]


@pytest.mark.parametrize("tokens,cols,pad", SIZES, ids=str)
@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("form", ["plain", "post", "gates"])
def test_norm(tokens, cols, pad, kind, form):
    dg = require_gpu()
    gate = {"plain": None, "post": "column", "gates": "token"}[form]
    residual, post, bias = form != "plain", form == "post", form == "gates"
    y, h = rows_of(tokens, cols, 11), rows_of(tokens, cols, 12) if residual else None
    par = parameters(tokens, cols, 13, gate, bias, post)
    opts = dict(post=post, kind=kind, eps=1e-5, res_scale=float(np.float32(0.7)))
    want = block.block_norm(bf16_to_f64(y), None if h is None else bf16_to_f64(h), **par, **opts)
    dev_par = {k: f32(v) for k, v in par.items()}
    th = None if h is None else padded(h, pad)
    r, x = empty_rows(tokens, cols, pad), empty_rows(tokens, cols, pad)
    dg.dg_block_norm(padded(y, pad), h=th, r=r, x=x, **dev_par, **opts)
    check_rows(r, want[0], want[2], "r")
    check_rows(x, want[1], want[3], "x")
    assert pads_kept(r) and pads_kept(x)
    # Each result alone is the same.
    r2, x2 = empty_rows(tokens, cols), empty_rows(tokens, cols)
    without = {k: v for k, v in dev_par.items() if k not in ("weight", "bias")}
    dg.dg_block_norm(padded(y, pad), h=th, r=r2, **without, **opts)
    dg.dg_block_norm(padded(y, pad), h=th, x=x2, **dev_par, **opts)
    assert torch.equal(r2, r) and torch.equal(x2, x)
    if cols % 128 == 0:
        for ue in (False, True):
            q, sf = code_buffers(tokens, cols, (tokens + 3) // 4 * 4 + 4, ue)
            r2 = empty_rows(tokens, cols)
            (dg.dg_block_norm_ue8m0 if ue else dg.dg_block_norm)(padded(y, pad), h=th, r=r2, q=q, sf=sf, **dev_par, **opts)
            assert torch.equal(r2, r)
            check_row_codes(q, sf, want[1], want[3], ue, "codes")


def test_norm_without_parameters_and_in_place():
    dg = require_gpu()
    y, h = rows_of(20, 1152, 21), rows_of(20, 1152, 22)
    stream = dev(h)
    x = empty_rows(20, 1152)
    dg.dg_block_norm(dev(y), h=stream, r=stream, x=x, post=True, kind="layer", eps=1e-5)
    want = block.block_norm(bf16_to_f64(y), bf16_to_f64(h), post=True, kind="layer", eps=1e-5)
    check_rows(stream, want[0], want[2], "r")
    check_rows(x, want[1], want[3], "x")


@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_zero_rows_and_zero_tiles_have_zero_codes(kind):
    dg = require_gpu()
    y = synth.bf16_normal((4, 256), 5)
    y[0], y[2, :128] = 0, 0
    if kind == "layer":
        y[0] = 0x4049  # a constant row: nothing but its mean (a sum of 256 equal values is exact)
    q, sf = code_buffers(4, 256, 4)
    dg.dg_block_norm(dev(y), q=q, sf=sf, kind=kind, eps=1e-5)
    assert np.all(host(q)[0] & 0x7F == 0) and np.all(host(sf)[:, 0] == 0)
    if kind == "rms":
        assert np.all(host(q)[2, :128] & 0x7F == 0) and host(sf)[0, 2] == 0 and host(sf)[1, 2] > 0


def test_values_that_are_not_finite_stay_in_their_row():
    dg = require_gpu()
    y = synth.bf16_normal((6, 2048), 6)
    clean = empty_rows(6, 2048)
    dg.dg_block_norm(dev(y), x=clean)
    y[1, 5], y[3, 2047], y[4, 0] = 0x7FC0, 0x7F80, 0xFF80
    x = empty_rows(6, 2048)
    dg.dg_block_norm(dev(y), x=x)
    assert torch.equal(x[[0, 2, 5]], clean[[0, 2, 5]])
    got = bf16_to_f64(host(x))
    assert np.all(np.isnan(got[1])) and np.isnan(got[3, 2047]) and np.isnan(got[4, 0])


def test_small_rows_reach_eps():
    """Rows below eps are divided by its root, not by theirs."""
    dg = require_gpu()
    y = synth.bf16_normal((3, 512), 7, 2.0 ** -40)
    x = empty_rows(3, 512)
    dg.dg_block_norm(dev(y), x=x, eps=1e-6)
    want = block.block_norm(bf16_to_f64(y), eps=1e-6)
    check_rows(x, want[1], want[3], "x")
    assert np.abs(want[1]).max() < 1e-8


BWD = [(0, 64, 0), (1, 8, 0), (3, 40, 8), (1000, 128, 8), (333, 256, 0), (5, 512, 0), (9, 1000, 16), (1100, 136, 0), (130, 1024, 0), (257, 2048, 8),
       (4, 3584, 0), (7, 4104, 8), (300, 7168, 0), (2, 8200, 0), (3, 16384, 8), (770, 8200, 0), (300, 12288, 8), (520, 16384, 0)]


@pytest.mark.parametrize("tokens,cols,pad", BWD, ids=str)
@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("form", ["plain", "post", "gates", "stream"])
def test_norm_bwd(tokens, cols, pad, kind, form):
    dg = require_gpu()
    gate = {"plain": None, "post": "column", "gates": "token", "stream": "column"}[form]
    post, bias, with_dx, with_dr = form in ("post", "stream"), form == "gates", form != "stream", form != "plain"
    dx, dr, r, y = (rows_of(tokens, cols, s) for s in (31, 32, 33, 34))
    par = parameters(tokens, cols, 35, gate, False, post)
    if not with_dx:
        del par["weight"]
    opts = dict(post=post, kind=kind, eps=1e-5, res_scale=float(np.float32(0.7)))
    dev_par = {k: f32(v) for k, v in par.items()}
    out = {"dy": empty_rows(tokens, cols, pad), "dh": empty_rows(tokens, cols, pad)}
    nans = lambda *s: torch.full(s, float("nan"), device="cuda")
    if with_dx:
        out["dweight"] = nans(cols)
    if bias:
        out["dbias"] = nans(cols)
    if post:
        out["dpost_weight"] = nans(cols)
    if gate:
        out["dgate"] = torch.full_like(dev_par["gate"], float("nan"))
    args = dict(dx=padded(dx, pad) if with_dx else None, dr=padded(dr, pad) if with_dr else None,
                r=padded(r, pad) if with_dx else None, y=padded(y, pad) if post or gate else None)
    ws = workspace(dg.dg_get_block_norm_bwd_workspace_size(tokens, cols))
    dg.dg_block_norm_bwd(workspace=ws, **args, **out, **dev_par, **opts)
    if tokens == 0:
        for name in ("dweight", "dbias", "dpost_weight", "dgate"):
            assert name not in out or not out[name].any(), name  # NaN would be true
        return
    f = lambda v: bf16_to_f64(v)
    want = block.block_norm_bwd(f(dx) if with_dx else None, f(dr) if with_dr else None, f(r), f(y) if post or gate else None,
                                **par, **opts)
    for name, got in out.items():
        (check_rows if name in ("dy", "dh") else check_f32)(got, *want[name], name)
    assert pads_kept(out["dy"]) and pads_kept(out["dh"])
    # The same again, bit for bit, over another workspace's contents; and dy alone.
    again = {k: torch.zeros_like(v) for k, v in out.items()}
    dg.dg_block_norm_bwd(workspace=workspace(ws.numel(), 0xFF), **args, **again, **dev_par, **opts)
    for name in out:
        assert torch.equal(again[name], out[name]), name
    alone = empty_rows(tokens, cols)
    dg.dg_block_norm_bwd(alone, **args, **dev_par, **opts)
    assert torch.equal(alone, out["dy"])


def test_norm_on_another_stream_and_in_a_graph():
    dg = require_gpu()
    t, n = 77, 7168
    ys = [dev(rows_of(t, n, s)) for s in (41, 42, 43)]
    y, h, dr = ys[0].clone(), dev(rows_of(t, n, 44)), dev(rows_of(t, n, 45))
    par = dict(post=True, gate=f32(np.random.default_rng(1).standard_normal(n)), weight=f32(np.ones(n)))
    r, x, dy = (empty_rows(t, n) for _ in range(3))
    q, sf = code_buffers(t, n, 80)
    dw, dg_ = torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
    ws = workspace(dg.dg_get_block_norm_bwd_workspace_size(t, n))

    def step():
        dg.dg_block_norm(y, h=h, r=r, x=x, q=q, sf=sf, **par)
        dg.dg_block_norm_bwd(dy, dx=x, dr=dr, r=r, y=y, dweight=dw, dgate=dg_, workspace=ws, **par)
        return [v.clone() for v in (r, x, q, sf, dy, dw, dg_)]

    want = []
    for v in ys:
        y.copy_(v)
        want.append(step())
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
    for k in (0, 2, 1, 0):
        y.copy_(ys[k])
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want[k]):
            assert torch.equal(a, b)


def test_norm_of_many_tokens():
    """More rows than workgroups take in one turn (narrow rows: four a workgroup), checked at both ends."""
    dg = require_gpu()
    t, n = (1 << 22) + 5, 8
    y = torch.randn(t, n, device="cuda").bfloat16()
    x = torch.zeros_like(y)
    dg.dg_block_norm(y, x=x)
    for part in (slice(0, 3), slice(t - 7, t)):
        want = block.block_norm(y[part].double().cpu().numpy())
        check_rows(x[part].view(torch.int16), want[1], want[3], "x")
    assert bool((x.float().pow(2).mean(1) - 1).abs().max() < 0.02)


def test_exponents_next_to_powers_of_two():
    """Rows whose largest normalised value is 448 / 256 = 1.75 sit on the edge between two exponents."""
    dg = require_gpu()
    y = np.zeros((2, 128), dtype=np.float32)
    y[:, :2] = 1.75, 1.0
    y[1, 0] = 1.7578125  # a bf16 step up
    # rms rows: scaled back by a weight so that x is y again
    k = np.sqrt((y.astype(np.float64) ** 2).mean(1, keepdims=True) + 1e-6)
    for row in range(2):
        weight = f32(np.full(128, k[row, 0]))
        q, sf = code_buffers(1, 128, 4, True)
        dg.dg_block_norm_ue8m0(torch.as_tensor(y[row:row + 1], device="cuda").bfloat16(), q=q, sf=sf, weight=weight)
        check_exponents(host(sf)[:, :1], np.array([[y[row, 0]]], dtype=np.float64), np.array([[4.0]]), "row")
