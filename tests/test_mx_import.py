"""The package imports where torch was built without GPU support, and its build module runs there."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_import_needs_nothing_that_only_gpu_builds_of_torch_have():
    code = ("import torch\n"
            "for n in [n for n in dir(torch._C) if n.startswith('_cuda_')]: delattr(torch._C, n)\n"
            "import bit_gemm_nvfp4_amd as nv, bit_gemm_nvfp4_amd.build\n"
            "assert nv.mx_workspace_size(1, 128, 256, 12288) > 0\n")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
