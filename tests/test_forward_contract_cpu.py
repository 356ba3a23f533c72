"""What the forward's entry points promise before anything is launched: checked without a GPU."""
import os
import subprocess
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def sv():
    from speculative_decoding_verify_07_gb300 import build
    if not os.path.exists(build.LIB):
        build.build()
    from speculative_decoding_verify_07_gb300 import binding
    return binding


def test_the_binding_imports_under_a_torch_without_cuda(sv):
    """Its checks and host functions serve there as before."""
    code = ("import torch\n"
            "for name in [n for n in dir(torch._C) if n.startswith('_cuda_')]:\n"
            "    delattr(torch._C, name)\n"
            "from speculative_decoding_verify_07_gb300 import binding as sv\n"
            "assert sv.row_block(7, 2, 1) == (4, 7) and sv.recur_workspace_size(1, 1, 1) > 0\n")
    run = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert run.returncode == 0, run.stderr
