"""Calls of the transformer block's operators without rows (no GPU): matrices without
values may have no address, and every other argument is checked as in any call."""

import pytest

from tests.test_block_abi import FAKE, INVALID, MISALIGNED, SHAPE, call, dg

GEMMS = ["dg_fp8_gemm_nt_epilogue", "dg_fp8_gemm_nt_ue8m0_epilogue"]
EMPTY = [dict(m=0), dict(n=0)]


@pytest.mark.parametrize("name", GEMMS)
@pytest.mark.parametrize("empty", EMPTY, ids=str)
@pytest.mark.parametrize("kw,status", [
    (dict(act=4), INVALID), (dict(act=-1), INVALID), (dict(residual=FAKE + 8), MISALIGNED), (dict(pre=FAKE + 8), MISALIGNED),
    (dict(bias=FAKE + 2), MISALIGNED), (dict(ld_res=-8), INVALID), (dict(ld_pre=516), MISALIGNED), (dict(ld_res=1 << 61), None),
    (dict(k=500), SHAPE), (dict(lda=504), INVALID), (dict(ldd=-8), INVALID), (dict(ld_sfa=66), MISALIGNED), (dict(ld_dsf=66), MISALIGNED),
    (dict(a=FAKE + 8), MISALIGNED), (dict(dq=FAKE + 8), MISALIGNED), (dict(k=-128), INVALID)], ids=str)
def test_gemm_of_nothing_checks_its_arguments(name, empty, kw, status):
    got = call(name, **{**empty, **kw})
    if status is None:  # too large only where there are rows
        assert got == (0 if "m" in empty else SHAPE)
    else:
        assert got == status and dg.dg_get_last_error_string() != ""


@pytest.mark.parametrize("name", GEMMS)
def test_narrow_or_ragged_terms_of_no_rows(name):
    assert call(name, m=0, ld_res=504) == INVALID and call(name, m=0, ld_pre=504) == INVALID
    assert call(name, m=0, n=520, ldd=520, ld_res=520, ld_pre=520) == SHAPE  # codes of whole blocks only
    assert call(name, m=-1, n=0) == INVALID and call(name, m=0, n=-1) == INVALID


@pytest.mark.parametrize("name", GEMMS)
def test_gemm_of_nothing_needs_no_addresses(name):
    nulls = dict(a=0, sfa=0, d=0, residual=0, pre=0, dq=0)
    assert call(name, m=0, ld_sfa=0, ld_dsf=0, **nulls) == 0
    assert call(name, n=0, b=0, sfb=0, d=0, residual=0, pre=0, dq=0, dsf=0, bias=0) == 0
    assert call(name, m=0, n=0, ld_sfa=0, ld_dsf=0, b=0, sfb=0, bias=0, dsf=0, **nulls) == 0


@pytest.mark.parametrize("name", ["dg_block_norm", "dg_block_norm_ue8m0"])
def test_norm_of_no_tokens_needs_no_addresses(name):
    """What a caller's allocator gives for [0][cols] matrices is null, for scales [cols/128][ld] it is not."""
    nothing = dict(tokens=0, y=0, h=0, r=0, x=0, q=0, gate=0)
    assert call(name, **nothing) == 0
    assert call(name, **{**nothing, "gate_kind": 2}) == 0
    assert call(name, **nothing, sf=0) == 0
    assert call(name, **nothing, ld_sf=0) == 0
    # The rest is checked as in any call.
    assert call(name, **nothing, kind=2) == INVALID and call(name, **nothing, eps=0.0) == INVALID
    assert call(name, **nothing, cols=520, ld_y=520) == SHAPE and call(name, **nothing, ld_sf=66) == MISALIGNED
    assert call(name, **nothing, post=0) == INVALID and call(name, tokens=0, y=FAKE + 8) == MISALIGNED
    assert call(name, **nothing, ld_y=504) == INVALID and call(name, **nothing, weight=FAKE + 4) == MISALIGNED
