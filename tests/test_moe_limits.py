"""Sizes that a launch cannot take are refused on the host, before anything is
enqueued (no GPU): a grid dimension carries fewer than 2^32 threads."""

import pytest

from tests.test_moe_abi import SHAPE, call, dg

REACHES_THE_LAUNCH = -5  # without a device

LARGE = 1 << 19  # rows and columns: 2^24 tiles of 128 x 128


@pytest.mark.parametrize("name,kw", [
    ("dg_requant_t", dict(rows=LARGE, cols=LARGE, ld_sf=LARGE, ld_sft=LARGE)),
    ("dg_moe_combine_bwd", dict(m_total=LARGE, cols=LARGE, ld_dy=LARGE, ld_d=LARGE, ld_dsf=LARGE, ld_dsft=LARGE)),
    ("dg_moe_combine_bwd", dict(m_total=1 << 30, cols=128, ld_dsf=1 << 30)),  # 2^24 workgroups of 64 rows
], ids=str)
def test_refused(name, kw):
    assert call(name, **kw) == SHAPE
    assert "2^" in dg.dg_get_last_error_string()


@pytest.mark.skipif(dg.torch.cuda.is_available(), reason="the launches would run on fake addresses")
@pytest.mark.parametrize("name,kw", [
    ("dg_requant_t", dict(rows=LARGE - 128, cols=LARGE, ld_sf=LARGE, ld_sft=LARGE)),
    ("dg_moe_combine_bwd", dict(m_total=LARGE - 128, cols=LARGE, ld_dy=LARGE, ld_d=LARGE, ld_dsf=LARGE, ld_dsft=LARGE)),
    ("dg_swiglu_bwd", dict(m_total=LARGE, inter=LARGE, ld_hsf=LARGE, ld_dact=LARGE, ld_dsf=LARGE, ld_dsft=2 * LARGE, ld_asft=LARGE)),
], ids=str)
def test_still_taken(name, kw):
    assert call(name, **kw) == REACHES_THE_LAUNCH
