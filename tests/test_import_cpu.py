"""The package imports, and refuses with its own errors, where torch was built
without CUDA and has none of the private CUDA functions that the binding uses."""

import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SCRIPT = """
import torch
for name in [n for n in dir(torch._C) if n.startswith("_cuda_")]:
    delattr(torch._C, name)
import mixture_experts_ffn_topk_gb300 as moe
try:
    moe.moe_grouped_gemm(torch.zeros(4, 16), torch.zeros(3, dtype=torch.int32), torch.zeros(2, 8, 16))
except ValueError as e:
    print("refused:", e)
"""


def test_import_without_cuda_in_torch():
    r = subprocess.run([sys.executable, "-c", SCRIPT], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    assert r.stdout.startswith("refused: tensors passed to the C ABI must live on a CUDA device")
