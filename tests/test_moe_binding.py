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
