"""The package imports with a torch that lacks the GPU's private functions (a CPU build)."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_import_without_a_gpu_build_of_torch():
    code = ("import torch\n"
            "for name in ('_cuda_getCurrentRawStream', '_cuda_getDevice'):\n"
            "    delattr(torch._C, name)\n"
            "import scale_search_weights_amd as pkg\n"
            "print(pkg.nvfp4.__name__, pkg.kvcache.__name__)\n")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    assert r.stdout.split() == ["scale_search_weights_amd.nvfp4", "scale_search_weights_amd.kvcache"]
