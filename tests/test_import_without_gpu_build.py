"""The package on a PyTorch that was built without a GPU: it imports, and the calls that touch no device work."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# such a PyTorch has none of torch._C's functions for devices and streams
CODE = """
import torch
for name in [n for n in dir(torch._C) if n.startswith("_cuda_")]:
    delattr(torch._C, name)
import nvfp4_block_scaled_02_amd as nv
import nvfp4_block_scaled_02_amd.build
assert nv.mxfp4_gemm_plan(8192, 8192, 8192) == "tile256"
assert nv.mxfp4_linear_workspace_bytes(8, 64) == 512 and nv.mxfp4_moe_workspace_bytes(4, 8, 64, 64, 2) > 0
assert nv.linear_workspace_bytes(8, 64) > 0
try:
    nv.mxfp4_quantize(torch.zeros(4, 64, dtype=torch.bfloat16))
except ValueError as e:
    assert "HIP device" in str(e)
else:
    raise AssertionError("a host tensor was taken")
print("ok")
"""


def test_import_and_host_only_calls():
    r = subprocess.run([sys.executable, "-c", CODE], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("ok"), r.stderr[-2000:]
