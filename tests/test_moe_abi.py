"""C-ABI checks of the mixture-of-experts operators that need no GPU: every
entry point include/dg_moe.h declares is exported and bound, and arguments
that break its rules are refused on the host, with a message, before anything
is enqueued."""

import ctypes
import os
import re
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "dg_moe.h")

dg = pytest.importorskip("moe_grouped_gemm_02_amd", reason="libdg.so not built")
from moe_grouped_gemm_02_amd import moe as binding  # noqa: E402

FAKE = 1 << 20  # an aligned non-null address; never dereferenced here
INVALID, SHAPE, MISALIGNED, WORKSPACE = -1, -2, -3, -4


def declarations():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    out = {}
    for name, args in re.findall(r"(?:int|size_t)\s+(dg_\w+)\s*\(([^)]*)\)\s*;", text):
        params = [a.strip().rsplit(" ", 1) for a in " ".join(args.split()).split(",")]
        out[name] = [(t + "*" * n.startswith("*"), n.lstrip("*")) for t, n in params]
    return out


DECLS = declarations()


def test_every_declared_entry_point_is_exported_and_bound():
    out = subprocess.run(["nm", "-D", "--defined-only", dg.LIB_PATH], capture_output=True, text=True, check=True).stdout
    exported = set(re.findall(r"\bT (dg_[a-z0-9_]+)$", out, flags=re.M))
    assert set(DECLS) <= exported and set(DECLS) == set(binding.EXPORTED)
    for name in DECLS:
        assert callable(getattr(dg, name)) and getattr(dg, name).__module__ == binding.__name__
        assert len(binding._SIGNATURES[name][1]) == len(DECLS[name])


VALID = dict(
    tokens=64, experts=256, topk=8, ld_logits=256, ld_dlogits=256, score=1, expert_groups=8, topk_groups=4, group_top=2,
    renormalize=1, scale=1.0, first_expert=0, num_groups=4, m_total=1024, m_max=256, cols=512, rows=256, ld_x=512, ld_sf=1024,
    total_rows=1024, ld_d=512, ld_y=512, ld_dy=512, ld_dsf=1024, ld_dsft=1024, ld_asft=512, ld_h=1024, ld_hsf=1024, ld_dact=512, inter=512,
    ld_sft=512, workspace_bytes=1 << 40, stream=None)


def call(name, **kw):
    args = []
    for ctype, pname in DECLS[name]:
        v = kw[pname] if pname in kw else VALID[pname] if pname in VALID else FAKE
        if pname == "masked_m" and "swiglu" in name and pname not in kw:
            v = None
        if pname == "m_indices" and "swiglu_quant" in name and pname not in kw:
            v = None
        args.append(ctypes.c_void_p(v) if "*" in ctype else v)
    return getattr(dg.raw(), name)(*args)


BAD = [
    ("dg_moe_route", dict(tokens=-1), INVALID), ("dg_moe_route", dict(experts=0), INVALID),
    ("dg_moe_route", dict(experts=1032, ld_logits=1032), SHAPE), ("dg_moe_route", dict(topk=0), INVALID),
    ("dg_moe_route", dict(topk=33), SHAPE), ("dg_moe_route", dict(experts=8, topk=9, expert_groups=1, topk_groups=1), INVALID),
    ("dg_moe_route", dict(ld_logits=255), INVALID), ("dg_moe_route", dict(ld_logits=1 << 60), SHAPE),
    ("dg_moe_route", dict(score=2), INVALID), ("dg_moe_route", dict(expert_groups=7), INVALID),
    ("dg_moe_route", dict(expert_groups=0), INVALID), ("dg_moe_route", dict(expert_groups=128), SHAPE),
    ("dg_moe_route", dict(topk_groups=0), INVALID), ("dg_moe_route", dict(topk_groups=9), INVALID),
    ("dg_moe_route", dict(group_top=3), INVALID), ("dg_moe_route", dict(logits=0), INVALID),
    ("dg_moe_route", dict(ids=0), INVALID), ("dg_moe_route", dict(weights=0), INVALID),
    ("dg_moe_route", dict(logits=FAKE + 2), MISALIGNED), ("dg_moe_route", dict(bias=FAKE + 2), MISALIGNED),
    ("dg_moe_route_bf16", dict(logits=FAKE + 1), MISALIGNED), ("dg_moe_route", dict(tokens=2**31 - 1), SHAPE),
    ("dg_moe_route_bwd", dict(ld_dlogits=255), INVALID), ("dg_moe_route_bwd", dict(dweights=0), INVALID),
    ("dg_moe_route_bwd_bf16", dict(dlogits=FAKE + 1), MISALIGNED),
    ("dg_moe_plan_contiguous", dict(m_total=1000), SHAPE), ("dg_moe_plan_contiguous", dict(num_groups=0), INVALID),
    ("dg_moe_plan_contiguous", dict(num_groups=1025), SHAPE), ("dg_moe_plan_contiguous", dict(first_expert=-1), INVALID),
    ("dg_moe_plan_contiguous", dict(k_offsets=0), INVALID), ("dg_moe_plan_contiguous", dict(m_indices=0), INVALID),
    ("dg_moe_plan_contiguous", dict(src=FAKE + 1), MISALIGNED),
    ("dg_moe_plan_contiguous", dict(tokens=1 << 20, workspace_bytes=15), WORKSPACE),
    ("dg_moe_plan_contiguous", dict(tokens=1 << 20, workspace=FAKE + 4), MISALIGNED),
    ("dg_moe_plan_masked", dict(m_max=-1), INVALID), ("dg_moe_plan_masked", dict(m_max=1 << 29), SHAPE),
    ("dg_moe_plan_masked", dict(masked_m=0), INVALID), ("dg_moe_plan_masked", dict(tokens=1 << 20, workspace=0), WORKSPACE),
    ("dg_moe_dispatch", dict(cols=500), SHAPE), ("dg_moe_dispatch", dict(cols=1 << 23, ld_x=1 << 23), SHAPE),
    ("dg_moe_dispatch", dict(ld_x=504), INVALID), ("dg_moe_dispatch", dict(ld_x=516), MISALIGNED),
    ("dg_moe_dispatch", dict(ld_sf=252), INVALID), ("dg_moe_dispatch", dict(ld_sf=1026), MISALIGNED),
    ("dg_moe_dispatch", dict(src=0), INVALID), ("dg_moe_dispatch_ue8m0", dict(q=FAKE + 8), MISALIGNED),
    ("dg_moe_dispatch", dict(num_groups=1 << 23, rows=1024), SHAPE),
    ("dg_moe_combine", dict(cols=500, ld_d=512), SHAPE), ("dg_moe_combine", dict(total_rows=-1), INVALID),
    ("dg_moe_combine", dict(ld_y=500), INVALID), ("dg_moe_combine", dict(ld_d=516), MISALIGNED),
    ("dg_moe_combine", dict(y=0), INVALID), ("dg_moe_combine", dict(d=FAKE + 2), MISALIGNED),
    ("dg_moe_combine_bwd", dict(m_total=100), SHAPE), ("dg_moe_combine_bwd", dict(dqt=0), INVALID),
    ("dg_moe_combine_bwd", dict(ld_dsft=508), INVALID), ("dg_moe_combine_bwd", dict(ld_dsf=1020), INVALID),
    ("dg_moe_combine_bwd", dict(workspace_bytes=1024 * 4 * 4 - 1), WORKSPACE), ("dg_moe_combine_bwd", dict(dweights=0), INVALID),
    ("dg_swiglu_quant", dict(inter=100, ld_h=200), SHAPE), ("dg_swiglu_quant", dict(ld_h=1016), INVALID),
    ("dg_swiglu_quant", dict(hsf=0), INVALID), ("dg_swiglu_quant", dict(ld_hsf=252), INVALID),
    ("dg_swiglu_quant", dict(m_indices=FAKE), INVALID), ("dg_swiglu_quant", dict(m_indices=FAKE, masked_m=FAKE), INVALID),
    ("dg_swiglu_quant_ue8m0", dict(sf=FAKE + 4), MISALIGNED), ("dg_swiglu_quant_ue8m0", dict(num_groups=0), INVALID),
    ("dg_swiglu_bwd", dict(m_total=64), SHAPE), ("dg_swiglu_bwd", dict(ld_dact=508), INVALID),
    ("dg_swiglu_bwd", dict(ld_dsft=1020), INVALID), ("dg_swiglu_bwd", dict(aqt=0), INVALID),
    ("dg_swiglu_bwd", dict(dqt=0), INVALID), ("dg_swiglu_bwd", dict(inter=1 << 22, ld_dact=1 << 22, ld_dsft=1 << 23), SHAPE),
    ("dg_requant_t", dict(rows=2**31 - 128, cols=65535 * 128, ld_sf=2**31 - 128, ld_sft=65535 * 128), SHAPE),
    ("dg_swiglu_quant", dict(num_groups=65536, rows=4, ld_sf=4, ld_hsf=4), SHAPE),
    ("dg_requant_t", dict(rows=100), SHAPE), ("dg_requant_t", dict(cols=130), SHAPE),
    ("dg_requant_t", dict(ld_sft=508), INVALID), ("dg_requant_t", dict(ld_sf=258), MISALIGNED),
    ("dg_requant_t", dict(qt=0), INVALID), ("dg_requant_t", dict(sf=FAKE + 4), MISALIGNED),
]


@pytest.mark.parametrize("name,kw,status", BAD, ids=lambda v: str(v))
def test_refusals(name, kw, status):
    assert call(name, **kw) == status
    assert dg.dg_get_last_error_string() != ""


def test_calls_with_nothing_to_do_succeed_without_a_device():
    for name in ("dg_moe_route", "dg_moe_route_bf16", "dg_moe_route_bwd", "dg_moe_route_bwd_bf16", "dg_moe_dispatch",
                 "dg_moe_combine", "dg_moe_combine_bwd"):
        assert call(name, tokens=0) == 0, name
    assert call("dg_moe_dispatch", rows=0, ld_sf=0) == 0
    assert call("dg_swiglu_quant", rows=0) == 0
    assert call("dg_swiglu_bwd", m_total=0) == 0
    assert call("dg_requant_t", rows=0) == 0


@pytest.mark.skipif(torch.cuda.is_available(), reason="the launches would run on fake addresses")
def test_valid_arguments_reach_the_launch():
    for name in DECLS:
        if not name.startswith("dg_get_"):
            assert call(name) == -5, name


def test_workspace_sizes():
    assert dg.dg_get_moe_combine_bwd_workspace_size(1024, 512) == 1024 * 4 * 4
    assert dg.dg_get_moe_combine_bwd_workspace_size(0, 512) == 0
    assert dg.dg_get_moe_plan_workspace_size(-1, 8, 4) == 0 and dg.dg_get_moe_plan_workspace_size(10, 8, 2000) == 0
    assert dg.dg_get_moe_plan_workspace_size(1 << 20, 8, 256) >= 256 * 4


def test_binding_refuses_host_tensors_and_unknown_scores():
    x, ids, w = torch.zeros(4, 16), torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
    with pytest.raises(ValueError, match="device tensor"):
        dg.dg_moe_route(x, ids, w)
    with pytest.raises(TypeError):
        dg.dg_moe_route(None, ids, w)
    with pytest.raises(ValueError, match="score"):
        binding._score("relu")
