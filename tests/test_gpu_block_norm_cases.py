"""GPU norms fused with gate and residual, and their gradient: rows and forms beside those
of tests/test_gpu_block_norm.py; tolerances in tests/block_util.py where not given."""

import numpy as np
import pytest
import torch

from oracle import block
from tests.block_util import check_f32, check_rows, code_buffers, empty_rows, f32, padded, pads_kept, workspace
from tests.gpu_util import bf16_to_f64, dev, host, require_gpu
from tests.test_gpu_block_norm import BWD, parameters, rows_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("ue8m0", [False, True])
@pytest.mark.parametrize("gate", [None, (512,), (0, 1)], ids=str)
def test_no_tokens(ue8m0, gate):
    """An empty batch with every result, through tensors as torch makes them."""
    dg = require_gpu()
    empty = lambda: torch.empty(0, 512, dtype=torch.bfloat16, device="cuda")
    fn = dg.dg_block_norm_ue8m0 if ue8m0 else dg.dg_block_norm
    q, sf = code_buffers(0, 512, 4, ue8m0)
    keep = sf.clone()
    par = dict(weight=f32(np.ones(512)), bias=f32(np.ones(512)), gate=None if gate is None else torch.zeros(gate, device="cuda"))
    fn(empty(), h=empty(), r=empty(), x=empty(), q=q, sf=sf, **par)
    fn(empty(), x=empty(), **par)
    fn(empty(), q=q, sf=sf, **par)
    assert torch.equal(sf, keep)


# Rows that are constant, or nearly, of 1000 (float32 numbers there are 2^-14 apart, bf16
# numbers 4): a mean that is off by a rounding would stay in every value, and be divided by
# the root of eps (0.06 for eps = 1e-6).  With the mean corrected by that of what it leaves,
# that is off by at most 2^-20 of a rounding of the sum (2^-18 of 1000), 2^-28 here, and
# 2^-18 after the division: OFF.  Everything else is relative: 2^-16 of the value (mean of
# squares, root, products), then one rounding to bf16.
OFF, RELATIVE = 2.0 ** -16, 2.0 ** -16
FLAT = [(136, 0), (1000, 8), (1536, 0), (3584, 0), (7168, 0), (8200, 8), (12288, 0), (16384, 0)]


def flat_rows(cols, seed):
    """bf16 values: constant rows, one with a single value a step up, one with a few steps, one ordinary."""
    rng = np.random.default_rng(seed)
    v = np.full((6, cols), 1000.0)
    v[1] = -1.1015625
    v[2, cols // 2] += 4.0
    v[3] += 4.0 * rng.integers(-1, 2, cols)
    v[4] = 37.0
    v[5] = 1000.0 + 4.0 * rng.integers(-64, 65, cols)
    y = torch.as_tensor(v, device="cuda").bfloat16()
    return y, y.double().cpu().numpy()


def near(got, want, off, what, half=2.0 ** -8):
    got = got.double().cpu().numpy()
    bad = ~(np.abs(got - want) <= (half + RELATIVE) * np.abs(want) + off)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size}, first at {np.argwhere(bad)[0]}: {got[bad][0]} for {want[bad][0]}"


def strided(rows, cols, pad):
    return torch.zeros(rows, cols + pad, dtype=torch.bfloat16, device="cuda")[:, :cols]


@pytest.mark.parametrize("cols,pad", FLAT, ids=str)
@pytest.mark.parametrize("post", [False, True])
def test_layer_norm_of_flat_rows(cols, pad, post):
    dg = require_gpu()
    y, v = flat_rows(cols, cols)
    bias = np.random.default_rng(1).standard_normal(cols).astype(np.float32)
    x = strided(6, cols, pad)
    if not post:
        dg.dg_block_norm(y, x=x, bias=f32(bias), kind="layer", eps=1e-6)
        want = block.block_norm(v, kind="layer", eps=1e-6)[1]
        near(x, want + bias, OFF + RELATIVE * np.abs(want), "x")
        # A constant row of bf16 numbers has an exact sum: nothing but the bias is left, in codes too.
        if cols % 128 == 0:
            q, sf = code_buffers(6, cols, 8)
            dg.dg_block_norm(y, q=q, sf=sf, kind="layer", eps=1e-6)
            assert not (q[[0, 1, 4]] & 0x7F).any() and not sf[:, [0, 1, 4]].any()
    else:  # the norm after the block meets them; no second norm
        r = strided(6, cols, pad)
        dg.dg_block_norm(y, r=r, post=True, kind="layer", eps=1e-6)
        near(r, block.block_norm(v, post=True, kind="layer", eps=1e-6)[0], OFF, "r")
    # Constant rows that are no bf16 numbers: the residual sum of two constants.
    h = torch.full((3, cols), 612.0, dtype=torch.bfloat16, device="cuda")
    x = strided(3, cols, pad)
    dg.dg_block_norm(y[:1].expand(3, cols).contiguous(), h=h, x=x, res_scale=0.7, kind="layer", eps=1e-6)
    near(x, np.zeros((3, cols)), OFF, "x of sums")


@pytest.mark.parametrize("cols,pad", FLAT, ids=str)
@pytest.mark.parametrize("post", [False, True])
def test_layer_norm_gradient_of_flat_rows(cols, pad, post):
    """dy is rstd (g - mean g - n mean(g n)): what n is off by (OFF) counts once with the mean of |g n| and once with
    that of |g|."""
    dg = require_gpu()
    rows, v = flat_rows(cols, cols)
    dx = torch.randn(6, cols, generator=torch.Generator(device="cuda").manual_seed(cols), device="cuda").bfloat16()
    g = dx.double().cpu().numpy()
    dy, out = strided(6, cols, pad), torch.full((cols,), float("nan"), device="cuda")
    ws = workspace(dg.dg_get_block_norm_bwd_workspace_size(6, cols))
    if post:
        dg.dg_block_norm_bwd(dy, dr=dx, y=rows, post=True, dpost_weight=out, kind="layer", eps=1e-6, workspace=ws)
        want = block.block_norm_bwd(dr=g, y=v, post=True, kind="layer", eps=1e-6)
    else:
        dg.dg_block_norm_bwd(dy, dx=dx, r=rows, dweight=out, kind="layer", eps=1e-6, workspace=ws)
        want = block.block_norm_bwd(dx=g, r=v, kind="layer", eps=1e-6)
    mean, k = block.stats(v, "layer", 1e-6)
    n, size = np.abs((v - mean) * k), np.abs(g)
    off = k * (RELATIVE * (size + size.mean(1, keepdims=True)) + (OFF + RELATIVE * n) * ((size * n).mean(1, keepdims=True) + size.mean(1, keepdims=True)))
    near(dy, want["dy"][0], off, "dy")
    name = "dpost_weight" if post else "dweight"
    near(out, want[name][0], (size * (OFF + RELATIVE * n)).sum(0), name, 2.0 ** -24)


# Forms of the gradient beside those of test_gpu_block_norm.py: two norms without the sums of a bias or of a column
# gate, with a bias, and a column gate without a norm after the block.
FORMS = {"post": (True, None, False), "post_token": (True, "token", False), "post_bias": (True, None, True), "post_all": (True, "column", True),
         "column": (False, "column", False), "column_bias": (False, "column", True)}


@pytest.mark.parametrize("tokens,cols,pad", [t for t in BWD if t[0]], ids=str)
@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("form", FORMS)
def test_gradient_of_other_forms(tokens, cols, pad, kind, form):
    dg = require_gpu()
    post, gate, bias = FORMS[form]
    dx, dr, r, y = (rows_of(tokens, cols, s) for s in (51, 52, 53, 54))
    par = parameters(tokens, cols, 55, gate, False, post)
    opts = dict(post=post, kind=kind, eps=1e-5, res_scale=float(np.float32(0.7)))
    dev_par = {k: f32(v) for k, v in par.items()}
    nans = lambda: torch.full((cols,), float("nan"), device="cuda")
    out = {"dy": empty_rows(tokens, cols, pad), "dh": empty_rows(tokens, cols, pad), "dweight": nans()}
    if bias:
        out["dbias"] = nans()
    if post:
        out["dpost_weight"] = nans()
    if gate:
        out["dgate"] = torch.full_like(dev_par["gate"], float("nan"))
    args = {k: padded(v, pad) for k, v in (("dx", dx), ("dr", dr), ("r", r), ("y", y))}
    ws = workspace(dg.dg_get_block_norm_bwd_workspace_size(tokens, cols))
    dg.dg_block_norm_bwd(workspace=ws, **args, **out, **dev_par, **opts)
    want = block.block_norm_bwd(*(bf16_to_f64(v) for v in (dx, dr, r, y)), **par, **opts)
    for name, got in out.items():
        (check_rows if name in ("dy", "dh") else check_f32)(got, *want[name], name)
    assert pads_kept(out["dy"]) and pads_kept(out["dh"])
    again = {k: torch.zeros_like(v) for k, v in out.items()}
    dg.dg_block_norm_bwd(workspace=workspace(ws.numel(), 0xFF), **args, **again, **dev_par, **opts)
    for name in out:
        assert torch.equal(again[name], out[name]), name


@pytest.mark.parametrize("cols", [136, 512, 7168])
@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_nan_stays_in_its_row(cols, kind):
    """Of the values, and of the gradient in its row and in the sums of its column."""
    dg = require_gpu()
    y, r, dx = (rows_of(5, cols, s) for s in (61, 62, 63))
    opts = dict(post=True, kind=kind, eps=1e-5)

    def run():
        x, dy = empty_rows(5, cols), empty_rows(5, cols)
        dg.dg_block_norm(dev(y), x=x, **opts)
        dw, dpw = torch.zeros(cols, device="cuda"), torch.zeros(cols, device="cuda")
        dg.dg_block_norm_bwd(dy, dx=dev(dx), r=dev(r), y=dev(y), dweight=dw, dpost_weight=dpw, **opts,
                             workspace=workspace(dg.dg_get_block_norm_bwd_workspace_size(5, cols)))
        return [t.clone() for t in (x, dy, dw, dpw)]

    clean = run()
    y[3, 7] = 0x7FC0
    got = run()
    keep = [0, 1, 2, 4]
    assert torch.equal(got[0][keep], clean[0][keep]) and torch.equal(got[1][keep], clean[1][keep]) and torch.equal(got[2], clean[2])
    assert np.isnan(bf16_to_f64(host(got[0])[3])).all() and np.isnan(bf16_to_f64(host(got[1])[3])).all() and bool(got[3].isnan().all())
    y[3, 7], dx[1, 9] = 0x3F80, 0xFFC0
    got = run()
    assert np.isnan(bf16_to_f64(host(got[1])[1])).all() and bool(got[2].isnan()[9]) and int(got[2].isnan().sum()) == 1
