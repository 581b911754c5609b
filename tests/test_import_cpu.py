"""The package on a torch built without GPU support: it imports, and the calls
that need no GPU work."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = """
import torch
for name in [n for n in dir(torch._C) if n.startswith("_cuda_")]:
    delattr(torch._C, name)
import boolean_weight_amd as bw
d = bw.mbok_desc_init(256, 512, 2)
assert bw.mbok_packed_bytes(d) > 0
assert bw.mbok_gemmt_workspace_bytes(d, 16) > 0
x = torch.zeros(4, 512, dtype=torch.bfloat16)
try:
    bw.mbok_gemmt(d, x, x, x)
except ValueError as e:
    assert "GPU" in str(e)
else:
    raise AssertionError("a host tensor was taken")
print("ok")
"""


def test_import_without_gpu_support():
    r = subprocess.run([sys.executable, "-c", PROGRAM], cwd=ROOT, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stderr[-2000:]
