"""The workspace of spec_scan, which needs no GPU: its size for every legal batch."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def sv():
    from speculative_decoding_verify_07_gb300 import build
    if not os.path.exists(build.LIB):
        build.build()
    from speculative_decoding_verify_07_gb300 import binding
    return binding


def test_an_empty_batch_has_a_workspace(sv):
    """(In a process of its own: a division by zero would end this one.)"""
    run = subprocess.run([sys.executable, "-c", "from speculative_decoding_verify_07_gb300 import binding as sv\n"
                          "for T in (0, 1, 17, 8192, 0x7fffff00):\n"
                          "    for N in (8, 16, 128):\n"
                          "        assert sv.LIB.spec_scan_workspace_size(0, T, 64, N) >= 256\n"
                          "assert sv.new_scan_workspace(0, 8192, 64, 16, 'cpu').numel() >= 256\n"], cwd=ROOT)
    assert run.returncode == 0
