"""The binding of the mixture-of-experts operators without a GPU: what it needs
of torch, and which workspaces it hands to the library."""

import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

pytest.importorskip("moe_grouped_gemm_02_amd", reason="libdg.so not built")

PROGRAM = """
import torch
if hasattr(torch._C, "_cuda_getCurrentRawStream"):
    del torch._C._cuda_getCurrentRawStream
import moe_grouped_gemm_02_amd as dg
from moe_grouped_gemm_02_amd import moe

class Stream:
    cuda_stream = 1234

torch.cuda.current_stream = lambda device=None: Stream()

class Tensor:
    device = "cuda:0"
    def get_device(self):
        return 0

assert moe._stream(Tensor()) == 1234
print("imported", len(moe.EXPORTED))
"""


def test_import_without_torch_private_stream_call():
    """The faster way to a stream's handle is a private name of torch: without it the public one serves."""
    res = subprocess.run([sys.executable, "-c", PROGRAM], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert res.returncode == 0 and "imported 16" in res.stdout, res.stderr[-2000:]


def test_workspaces_are_device_tensors():
    """A kernel writes its workspace: host memory is refused like any other host tensor, and
    so is what only looks as large as it says."""
    import torch
    from moe_grouped_gemm_02_amd import moe
    assert moe._workspace(None) == (None, 0)
    with pytest.raises(ValueError, match="device tensor"):
        moe._workspace(torch.zeros(64, dtype=torch.uint8))
    with pytest.raises(TypeError, match="torch.Tensor"):
        moe._workspace(1 << 20)


@pytest.mark.gpu
def test_calls_refuse_other_workspaces():
    import torch
    from tests.gpu_util import require_gpu
    dg = require_gpu()
    ids = torch.zeros(8192, 1, dtype=torch.int32, device="cuda")
    rows, src, count = torch.empty_like(ids), torch.empty(8192, dtype=torch.int32, device="cuda"), ids[:1, 0].clone()
    size = dg.dg_get_moe_plan_workspace_size(8192, 1, 1)
    spread = torch.zeros(1, dtype=torch.uint8, device="cuda").expand(size)
    for ws in (torch.zeros(size, dtype=torch.uint8), spread):
        with pytest.raises(ValueError):
            dg.dg_moe_plan_masked(ids, rows, src, count, workspace=ws)
        with pytest.raises(ValueError):
            dg.dg_moe_plan_contiguous(ids, rows, src, torch.empty_like(src), torch.zeros(2, dtype=torch.int32, device="cuda"), workspace=ws)
    dy = torch.zeros(1, 128, dtype=torch.bfloat16, device="cuda")
    d, dq = torch.zeros(128, 128, dtype=torch.bfloat16, device="cuda"), torch.zeros(128, 128, dtype=torch.uint8, device="cuda")
    w = torch.zeros(1, 1, device="cuda")
    with pytest.raises(ValueError):
        dg.dg_moe_combine_bwd(dy, d, src[:128], ids[:1], w, dq, torch.zeros(1, 128, device="cuda"), None, None, w.clone(),
                              workspace=torch.zeros(512, dtype=torch.uint8))


@pytest.mark.gpu
def test_sizes_past_32_bits_are_refused():
    """Sizes go to the library as 32-bit numbers: 2^32 + 5 must not arrive as 5."""
    import torch
    from tests.gpu_util import require_gpu
    dg = require_gpu()
    n = 2 ** 32 + 5
    long = torch.empty(n, dtype=torch.bfloat16, device="cuda")
    few = torch.zeros(5, 1, dtype=torch.int32, device="cuda")
    ids, w = torch.empty(n, 1, dtype=torch.int32, device="cuda"), torch.empty(n, 1, device="cuda")
    with pytest.raises(ValueError, match="2\\^31"):
        dg.dg_moe_route_bf16(long.view(n, 1), ids, w)
    with pytest.raises(ValueError, match="2\\^31"):
        dg.dg_moe_combine(long.view(1, n), few[:1], long.view(1, n))
    with pytest.raises(ValueError, match="2\\^31"):
        dg.dg_moe_plan_masked(few, few.clone(), ids.view(-1), few[:1, 0].clone())
    with pytest.raises(ValueError, match="2\\^31"):
        dg.dg_moe_plan_masked(ids, ids, few[:, 0].clone(), few[:1, 0].clone())
    with pytest.raises(ValueError, match="2\\^31"):
        dg.dg_swiglu_quant(long.view(1, 1, n), long[:2 ** 31].view(torch.uint8).view(1, 1, 2 ** 32), w.view(-1)[:2 ** 27].view(1, 2 ** 25, 4))
    x, sf = torch.zeros(8, 128, dtype=torch.bfloat16, device="cuda"), torch.zeros(1, 8, device="cuda")
    src, q = torch.zeros(8, dtype=torch.int32, device="cuda"), torch.zeros(8, 128, dtype=torch.uint8, device="cuda")
    with pytest.raises(ValueError, match="2\\^31"):
        dg.dg_moe_dispatch(x, src, q, sf, topk=2 ** 32 + 1)
    with pytest.raises(ValueError, match="2\\^31"):
        dg.dg_moe_plan_masked(few, few.clone(), src, few[:1, 0].clone(), first_expert=2 ** 32)
    with pytest.raises(ValueError, match="2\\^31"):
        dg.dg_moe_route(torch.zeros(5, 8, device="cuda"), few, torch.zeros(5, 1, device="cuda"), expert_groups=2 ** 32 + 2)
