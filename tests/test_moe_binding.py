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
