"""The workspace of spec_scan, which needs no GPU: its size for every legal batch."""
import ctypes
import os
import random
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


# Through the source's own arithmetic: the most bytes that any number of groups takes of a workspace, and how many parts.
PROBE = """
#include "spec_scan_split.h"
using namespace specv;
extern "C" size_t used(int B, int T, int D, int N, int groups) {
  const ScanSplit W = scan_split(B, T, D, D / groups, N);
  return scan_bytes(scan_parts(W, B), D, N);
}
extern "C" size_t most_used(int B, int T, int D, int N) {
  size_t most = 0;
  for (int g = 1; g <= D; ++g)
    if (D % g == 0) most = std::max(most, used(B, T, D, N, g));
  return most;
}
"""


@pytest.fixture(scope="module")
def split(tmp_path_factory):
    from speculative_decoding_verify_07_gb300 import build
    path = tmp_path_factory.mktemp("scan")
    (path / "probe.cpp").write_text(PROBE)
    subprocess.run(["g++", "-std=c++17", "-O2", "-shared", "-fPIC", "-I", build.CSRC, "-o", str(path / "probe.so"), str(path / "probe.cpp")],
                   check=True)
    lib = ctypes.CDLL(str(path / "probe.so"))
    lib.used.restype = lib.most_used.restype = ctypes.c_size_t
    return lib


# (B, T, D, N, groups): fewer CTAs and more parts with several groups than with one
GROUPED = [(8, 2048, 512, 8, 8), (9, 8192, 64, 16, 2), (17, 4096, 64, 16, 2), (5, 1279, 384, 32, 8), (7, 2934, 312, 16, 2),
           (2, 1551, 1338, 16, 2), (8, 1536, 576, 8, 2), (1, 2048, 1728, 16, 36)]


@pytest.mark.parametrize("B,T,D,N,groups", GROUPED)
def test_groups_that_divide_otherwise_than_one(sv, split, B, T, D, N, groups):
    assert split.used(B, T, D, N, groups) > split.used(B, T, D, N, 1)
    assert split.used(B, T, D, N, groups) <= sv.LIB.spec_scan_workspace_size(B, T, D, N)


def test_no_call_takes_more_than_the_workspace(sv, split):
    rng = random.Random(1)
    log = lambda lo, hi: int(lo * (hi / lo) ** rng.random() + 0.5)
    split_calls = 0
    for i in range(20000):
        B, T, N = log(1, 400), log(1, 0x7fffff00) if i % 4 == 0 else log(1, 40000), rng.choice([8, 16, 32, 64, 128])
        D = rng.randrange(1, 65) * rng.choice([1, 2, 6, 8, 16, 48, 64]) if i % 2 else log(1, 16384)
        most = split.most_used(B, T, D, N)
        split_calls += most > 0
        assert most <= sv.LIB.spec_scan_workspace_size(B, T, D, N), (B, T, D, N)
    assert split_calls > 2000


def test_a_workspace_serves_smaller_batches_and_shorter_rows(sv, split):
    size = sv.LIB.spec_scan_workspace_size
    assert split.used(1, 2048, 4096, 16, 1) > 256          # a batch that is split, where a larger one is not
    assert size(4, 2048, 4096, 16) >= split.used(1, 2048, 4096, 16, 1)
    rng = random.Random(2)
    for N in (8, 16, 32, 64, 128):
        for _ in range(200):
            D, T = rng.randrange(1, 8192), rng.randrange(1, 20000)
            rows = [0] + sorted(rng.sample(range(1, 400), 8)) + [65535]
            tokens = sorted({rng.randrange(0, T + 1) for _ in range(6)} | {0, 1, T})
            by_rows, by_tokens = [size(b, T, D, N) for b in rows], [size(3, t, D, N) for t in tokens]
            assert by_rows == sorted(by_rows) and by_tokens == sorted(by_tokens), (D, T, N)
            most = max(split.most_used(b, t, D, N) for b in rows[1:4] for t in tokens[-3:])
            assert most <= size(rows[3], T, D, N), (D, T, N)
