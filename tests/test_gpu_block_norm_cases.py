"""GPU norms fused with gate and residual, and their gradient: rows and forms beside those
of tests/test_gpu_block_norm.py; tolerances in tests/block_util.py where not given."""

import numpy as np
import pytest
import torch

from tests.block_util import code_buffers, f32
from tests.gpu_util import require_gpu

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
