"""The binding imports on a torch build without GPU support, whose ``torch._C``
has no stream and device accessors. No GPU."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_imports_without_torchs_gpu_accessors():
    code = """
import torch
for name in ("_cuda_getDevice", "_cuda_getCurrentRawStream"):
    if hasattr(torch._C, name):
        delattr(torch._C, name)
import draft_verify_sampling_spec_amd as d
assert d.binding.spec_verify_cache_bytes(3, 2, 128, 64) == 3 * 2 * 2 * 34 * 128
"""
    res = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert res.returncode == 0, res.stderr[-2000:]
