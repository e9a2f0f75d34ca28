"""GPU mixture-of-experts calls along paths that small shapes do not take."""

import numpy as np
import pytest
import torch

import synth
from oracle import moe
from tests.gpu_util import bf16_to_f64, dev, host, require_gpu
from tests.test_gpu_moe_exchange import FILL, check_transposed

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
