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


def calls(sv):
    """Each call on well-formed arguments that lie on the host, with what else it is given."""
    kv = torch.zeros((5, 2, 16, 64), dtype=torch.bfloat16)
    cu, ln, table = torch.tensor([0, 1, 2], dtype=torch.int32), torch.ones(2, dtype=torch.int32), torch.zeros((2, 3), dtype=torch.int32)
    q, new, g = torch.zeros((2, 8, 64), dtype=torch.bfloat16), torch.zeros((2, 2, 64), dtype=torch.bfloat16), torch.zeros((2, 3, 8))
    cache = (cu, ln, table, kv, kv.clone())
    return (lambda **kw: sv.spec_attend(q, *cache, max_tokens=1, **kw), lambda **kw: sv.spec_recur(g, g, **kw),
            lambda **kw: sv.spec_recur_backward(g, g, g, **kw), lambda **kw: sv.spec_cache_write(new, new, *cache, **kw),
            lambda **kw: sv.spec_cache_read(2, *cache, **kw))


def test_tensors_on_the_host_are_refused(sv):
    for call in calls(sv):
        with pytest.raises(ValueError, match="CUDA device"):
            call()


@pytest.mark.parametrize("unfit", [lambda n: torch.zeros(n // 4, dtype=torch.int32), lambda n: torch.zeros(2 * n, dtype=torch.uint8)[::2],
                                   lambda n: torch.zeros(1, dtype=torch.uint8).expand(n), lambda n: torch.zeros(n, dtype=torch.uint8, device="meta")])
def test_unfit_workspaces_are_refused(sv, unfit):
    for call in calls(sv)[:3]:
        with pytest.raises(ValueError, match="workspace"):
            call(workspace=unfit(1 << 26))


P, DIM, REACHED = 4096, -2, (-6, -7)      # a fake, aligned address: never dereferenced; without a GPU a valid call ends there
MOST = 0x7FFFFF00


@pytest.mark.parametrize("max_pages,page,ok", [(2 ** 31 - 1, 1, False), (MOST + 1, 1, False), (MOST, 1, True),
                                               (2 ** 31 // 24, 24, False), (MOST // 24, 24, True)])
@pytest.mark.skipif(torch.cuda.is_available(), reason="the calls would run")
def test_positions_stay_within_32_bits(sv, max_pages, page, ok):
    view = sv.CACHE_T.pack(P, P, 0, 0, P, P, P, 0, 0, 1, 1, max_pages, 5, 2, page, 64)
    codes = (sv.LIB.spec_attend(P, 0, 1, 4, 0.1, 1, view, P, P, None, P, 1 << 40, None),
             sv.LIB.spec_cache_write(P, P, 1, 0, 1, view, None, None), sv.LIB.spec_cache_read(P, P, 1, view, None, None))
    assert all(c in REACHED if ok else c == DIM for c in codes), codes


@pytest.mark.skipif(torch.cuda.is_available(), reason="the calls would run")
@pytest.mark.parametrize("T,ok", [(2 ** 31 - 1, False), (MOST + 1, False), (MOST, True)])
def test_a_rows_tokens_stay_within_32_bits(sv, T, ok):
    size = sv.LIB.spec_recur_workspace_size(1, T, 1)
    # three words of eight bytes for each of 64 channels of a tile of 64 tokens, behind a header of 256 bytes
    assert size == (256 + 3 * 8 * 64 * (T // 64) if ok else 0)
    codes = (sv.LIB.spec_recur(P, 0, 1, P, 0, 1, 1, None, None, 0, None, 1, T, 1, P, 1, None, None, 0, None, P, 1 << 50, None),
             sv.LIB.spec_recur_backward(P, 0, 1, P, 1, P, None, 1, None, None, 0, None, 1, T, 1, P, P, None, None, P, 1 << 50, None))
    assert all(c in REACHED if ok else c == DIM for c in codes), codes
