"""The package imports, and checks arguments, on a torch built without a GPU (no GPU needed)."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CODE = """
import torch
for name in [n for n in dir(torch._C) if n.startswith("_cuda_")]:
    delattr(torch._C, name)
import group_wise_affine_unpack_amd as qa
assert qa.lib().qaff_version() > 0
w = torch.zeros((2, 64), dtype=torch.bfloat16)
for call in (lambda: qa.quantize_pack_affine(w, 64, 4), lambda: qa.rmsnorm(w, w[0])):
    try:
        call()
    except ValueError as e:
        assert "GPU" in str(e), e
    else:
        raise AssertionError("a CPU tensor was taken")
print("imported")
"""


def test_import_without_the_gpu_names_of_torch():
    r = subprocess.run([sys.executable, "-c", CODE], capture_output=True, text=True, cwd=ROOT, timeout=300)
    assert r.returncode == 0 and "imported" in r.stdout, r.stderr[-2000:]
