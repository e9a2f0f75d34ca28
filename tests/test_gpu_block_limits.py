"""GPU operators of a transformer block on matrices of more than 4 GiB: rows behind
the 32-bit byte offsets come out as in a call on those rows alone, bit for bit (no
value of a row depends on the others where the call wants no sum over rows)."""

import pytest
import torch

from tests.block_util import workspace
from tests.gpu_util import require_gpu

pytestmark = pytest.mark.gpu

ROWS, COLS = 300 * 1024, 8192  # 4.7 GiB of bf16
LAST = 256


@pytest.fixture(autouse=True)
def release():
    yield
    torch.cuda.empty_cache()


def random_rows(rows, cols, seed):
    """bf16 rows that repeat every 4093, so that rows 2^32 bytes apart differ."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    part = torch.randn(4093, cols, generator=g, device="cuda").bfloat16()
    return part.repeat(-(-rows // 4093), 1)[:rows].contiguous()


def bf16(rows):
    return torch.full((rows, COLS), float("nan"), dtype=torch.bfloat16, device="cuda")


def codes(rows, cols):
    return torch.zeros(rows, cols, dtype=torch.uint8, device="cuda")


def test_norm_and_its_gradient():
    dg = require_gpu()
    y, h = random_rows(ROWS, COLS, 1), random_rows(ROWS, COLS, 2)
    r, q, sf = bf16(ROWS), codes(ROWS, COLS), torch.zeros(COLS // 128, ROWS, device="cuda")
    dg.dg_block_norm(y, h=h, r=r, q=q, sf=sf, res_scale=0.5)
    tail = slice(ROWS - LAST, ROWS)
    r1, q1, sf1 = bf16(LAST), codes(LAST, COLS), torch.zeros(COLS // 128, LAST, device="cuda")
    dg.dg_block_norm(y[tail], h=h[tail], r=r1, q=q1, sf=sf1, res_scale=0.5)
    assert torch.equal(r[tail], r1) and torch.equal(q[tail], q1) and torch.equal(sf[:, tail], sf1)
    del q, h
    dy, one = bf16(ROWS), bf16(LAST)
    dg.dg_block_norm_bwd(dy, dx=y, r=r)
    dg.dg_block_norm_bwd(one, dx=y[tail], r=r1)
    assert torch.equal(dy[tail], one)


def test_epilogue_and_its_gradient():
    dg = require_gpu()
    x = random_rows(ROWS, 128, 3)
    a, sfa = codes(ROWS, 128), torch.zeros(1, ROWS, device="cuda")
    dg.dg_quant_1x128(x, a, sfa)
    w = torch.randn(COLS, 128, device="cuda").bfloat16()
    b, sfb = codes(COLS, 128), torch.zeros(COLS // 128, 1, device="cuda")
    dg.dg_quant_128x128(w, b, sfb)
    residual, bias = random_rows(ROWS, COLS, 4), torch.randn(COLS, device="cuda")
    d, pre = bf16(ROWS), bf16(ROWS)
    ws = workspace(dg.dg_get_workspace_size(ROWS, COLS, 128))
    dg.dg_fp8_gemm_nt_epilogue(a, sfa, b, sfb, d, bias=bias, act="silu", residual=residual, pre=pre, workspace=ws.zero_())
    tail = slice(ROWS - LAST, ROWS)
    d1, pre1 = bf16(LAST), bf16(LAST)
    ws = workspace(dg.dg_get_workspace_size(LAST, COLS, 128))
    dg.dg_fp8_gemm_nt_epilogue(a[tail], sfa[:, tail].contiguous(), b, sfb, d1, bias=bias, act="silu", residual=residual[tail], pre=pre1,
                               workspace=ws.zero_())
    # One slice of K: the same sum in every tile.
    assert torch.equal(d[tail], d1) and torch.equal(pre[tail], pre1)
    del residual
    dq, dsf = codes(ROWS, COLS), torch.zeros(COLS // 128, ROWS, device="cuda")
    dqt, dsft = codes(COLS, ROWS), torch.zeros(ROWS // 128, COLS, device="cuda")
    dg.dg_epilogue_bwd(d, dq, dsf, pre=pre, act="silu", dqt=dqt, dsft=dsft)
    dq1, dsf1 = codes(LAST, COLS), torch.zeros(COLS // 128, LAST, device="cuda")
    dqt1, dsft1 = codes(COLS, LAST), torch.zeros(LAST // 128, COLS, device="cuda")
    dg.dg_epilogue_bwd(d1, dq1, dsf1, pre=pre1, act="silu", dqt=dqt1, dsft=dsft1)
    assert torch.equal(dq[tail], dq1) and torch.equal(dsf[:, tail], dsf1)
    assert torch.equal(dqt[:, tail], dqt1) and torch.equal(dsft[-(LAST // 128):], dsft1)


def test_balance_gradient():
    dg = require_gpu()
    tokens, experts = 1200 * 1024, 1024  # 4.7 GiB of float32
    logits = random_rows(tokens, experts, 5).float()
    ids = torch.randint(0, experts, (tokens, 2), dtype=torch.int32, device="cuda")
    counts, used = torch.zeros(2, experts, dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
    loss = torch.zeros(1, device="cuda")
    off = torch.tensor([0, tokens - LAST, tokens], dtype=torch.int32, device="cuda")
    dg.dg_moe_balance(logits, ids, counts, used, loss, seq_offsets=off, workspace=workspace(dg.dg_get_moe_balance_workspace_size(tokens, experts, 2)))
    tail = slice(tokens - LAST, tokens)
    assert torch.equal(counts[1], torch.bincount(ids[tail].flatten(), minlength=experts).int())
    assert used.tolist() == [tokens - LAST, LAST]
    out = torch.full_like(logits, float("nan"))
    dg.dg_moe_balance_bwd(logits, counts, used, out, 2, seq_offsets=off)
    one = torch.zeros(LAST, experts, device="cuda")
    # Half the loss each: a mean over one sequence has twice the gradient of a mean over two.
    dg.dg_moe_balance_bwd(logits[tail], counts[1:], used[1:], one, 2, coef=0.5)
    assert torch.equal(out[tail], one)
