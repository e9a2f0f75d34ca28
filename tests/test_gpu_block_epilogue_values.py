"""GPU epilogue of the dense GEMM and its gradient where values are not finite: NaN and
infinities of z, dd and the bias show where dg_block.h says, and nowhere else.
"""

import numpy as np
import pytest
import torch

from oracle import block
from synth import bf16_normal
from tests.block_util import check_f32, code_buffers, workspace
from tests.gpu_util import bf16_to_f64, dev, host, require_gpu

pytestmark = pytest.mark.gpu

ACTS = ["none", "relu", "silu", "gelu_tanh"]
NAN, QUIET, INF, MINUS_INF = 0x7FC0, 0xFFC1, 0x7F80, 0xFF80


def gradient(dg, dd, z, act):
    """(dq, dsf, dqt, dsft, dbias) on the host."""
    rows, cols = dd.shape
    dq, dsf = code_buffers(rows, cols, (rows + 3) // 4 * 4)
    tiles = -(-rows // 128)
    dqt, dsft = torch.zeros(cols, tiles * 128, dtype=torch.uint8, device="cuda"), torch.zeros(tiles, cols, device="cuda")
    db = torch.zeros(cols, device="cuda")
    dg.dg_epilogue_bwd(dev(dd), dq, dsf, pre=None if act == "none" else dev(z), act=act, dqt=dqt, dsft=dsft, dbias=db,
                       workspace=workspace(dg.dg_get_epilogue_bwd_workspace_size(rows, cols)))
    return [host(t) for t in (dq, dsf, dqt, dsft, db)]


def same_but_for(got, want, rows, cols):
    """Everything as in `want` but the codes' tiles and columns that the given values belong to."""
    keep_r = np.ones(len(want[0]), bool)
    keep_r[rows] = False
    keep_c = np.ones(want[0].shape[1], bool)
    keep_c[cols] = False
    assert np.array_equal(got[0][keep_r], want[0][keep_r]) and np.array_equal(got[1][:, :len(keep_r)][:, keep_r], want[1][:, :len(keep_r)][:, keep_r])
    assert np.array_equal(got[2][keep_c], want[2][keep_c]) and np.array_equal(got[3][:, keep_c], want[3][:, keep_c])
    assert np.array_equal(got[4][keep_c], want[4][keep_c])


@pytest.mark.parametrize("rows", [100, 200])
@pytest.mark.parametrize("act", ACTS)
def test_nan_shows_in_its_column_of_dbias(rows, act):
    """A NaN of z or of dd, of either sign, in one and in several tiles of rows."""
    dg = require_gpu()
    dd, z = bf16_normal((rows, 384), 1), bf16_normal((rows, 384), 2, 2.0)
    want = gradient(dg, dd, z, act)
    at_rows, at_cols = [5, rows - 1, 70], [7, 200, 383]
    for where in (("dd", "z") if act != "none" else ("dd",)):
        bad = {"dd": dd.copy(), "z": z.copy()}
        bad[where][at_rows, at_cols] = [NAN, QUIET, NAN]
        got = gradient(dg, bad["dd"], bad["z"], act)
        assert np.flatnonzero(np.isnan(got[4])).tolist() == at_cols, where
        same_but_for(got, want, at_rows, at_cols)


@pytest.mark.parametrize("act", ["relu", "silu", "gelu_tanh"])
def test_infinite_z_has_the_slopes_limit(act):
    dg = require_gpu()
    dd, z = bf16_normal((140, 256), 3), bf16_normal((140, 256), 4, 2.0)
    far = z.copy()
    z[[3, 130], [10, 11]], far[[3, 130], [10, 11]] = [INF, MINUS_INF], [0x7149, 0xF149]  # +-1e30
    got = gradient(dg, dd, z, act)
    for u, v in zip(got, gradient(dg, dd, far, act)):
        assert np.array_equal(u, v)
    v = bf16_to_f64(dd) * block.act_slope(bf16_to_f64(far), act)
    check_f32(torch.as_tensor(got[4]), v.sum(0), np.abs(v).sum(0) + np.abs(bf16_to_f64(dd)).sum(0), "dbias")


@pytest.mark.parametrize("act", ACTS)
def test_nan_of_a_bias_shows_in_its_column(act):
    dg = require_gpu()
    m, n = 70, 136
    a, b = torch.zeros(m, 128, dtype=torch.uint8, device="cuda"), torch.zeros(n, 128, dtype=torch.uint8, device="cuda")
    bias = torch.ones(n, device="cuda")
    bias[9], bias[135] = float("nan"), -float("nan")
    d, z = (torch.zeros(m, n, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    dg.dg_fp8_gemm_nt_epilogue(a, torch.zeros(1, 72, device="cuda"), b, torch.zeros(2, 1, device="cuda"), d, bias=bias, act=act, pre=z)
    nan = bias.isnan().expand(m, n)
    assert torch.equal(d.isnan(), nan) and torch.equal(z.isnan(), nan)


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_activations_down_to_the_last_bf16_numbers(act):
    """Where z / (1 + e^-t) leaves the range of bf16 (z = -88 to -98 for the SiLU, about -10 for the GELU), results are as
    accurate as elsewhere: t is off by a few roundings, 2^-22 of up to 142 (powers of 2), which is 2^-14.6 of the result;
    then one rounding, to half of 2^-133 at least."""
    dg = require_gpu()
    n = 4096
    z = torch.cat([torch.linspace(-100, -80, n // 2, device="cuda"), torch.linspace(-12, -8, n // 2, device="cuda")])
    d = torch.zeros(1, n, dtype=torch.bfloat16, device="cuda")
    a, b = torch.zeros(1, 0, dtype=torch.uint8, device="cuda"), torch.zeros(n, 0, dtype=torch.uint8, device="cuda")
    dg.dg_fp8_gemm_nt_epilogue(a, torch.zeros(0, 4, device="cuda"), b, torch.zeros(32, 0, device="cuda"), d, bias=z, act=act)
    want = block.act(z.double().cpu().numpy(), act)
    got = d[0].double().cpu().numpy()
    bad = ~(np.abs(got - want) <= (2.0 ** -8 + 2.0 ** -14.5) * np.abs(want) + 2.0 ** -134)
    assert not bad.any(), f"{bad.sum()}, first at z = {float(z[int(np.flatnonzero(bad)[0])])}: {got[bad][0]} for {want[bad][0]}"
    tiny = np.abs(want) < 2.0 ** -126  # some of them below the normal range
    assert 10 < (tiny & (want < -2.0 ** -133)).sum()


def test_gelu_slope_of_large_negative_z():
    """One row, so that dbias is dd times the slope in float32: down to z = -10 within what t is off by (2^-23 of up to
    126 powers of two, 2^-16, and as much again in the other factors), past that below 2^-117."""
    dg = require_gpu()
    z = np.concatenate([np.linspace(-10, -4, 384), np.linspace(-40, -10, 128)])
    zt = torch.as_tensor(z, device="cuda").bfloat16()[None]
    z = zt[0].double().cpu().numpy()
    dd = torch.ones(1, 512, dtype=torch.bfloat16, device="cuda")
    dq, dsf = code_buffers(1, 512, 4)
    db = torch.zeros(512, device="cuda")
    dg.dg_epilogue_bwd(dd, dq, dsf, pre=zt, act="gelu_tanh", dbias=db)
    got, want = host(db).astype(np.float64), block.act_slope(z, "gelu_tanh")
    near = z >= -10
    assert near.sum() > 380 and np.all(np.abs(got - want)[near] <= 2.0 ** -15 * np.abs(want)[near])
    assert np.all(np.abs(got[~near]) <= 2.0 ** -117)
