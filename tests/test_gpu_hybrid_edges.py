"""Edges of the causal convolution, the selective scan and the attention over a shared prefix on the GPU.

Tolerances count roundings: half a step of bf16 is 2^-8 relative, of float32 2^-24.
"""
import numpy as np
import pytest
import torch

from oracle import hybrid as oh
from tests.test_gpu_hybrid import F32, half, host, near

pytestmark = pytest.mark.gpu

DT = [torch.bfloat16, torch.float32]


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")


@pytest.mark.parametrize("T", [0, 3, 900])
def test_an_empty_batch(T):
    from speculative_decoding_verify_07_gb300 import binding as sv
    x, b = torch.empty((0, T, 24), device="cuda"), torch.empty((0, T, 1, 16), device="cuda")
    y, last = sv.spec_scan(x, x, torch.zeros((24, 16), device="cuda"), b, b)
    assert y.shape == (0, T, 24) and last.shape == (0, 24, 16)
    y, last = sv.spec_conv(x, torch.ones((4, 24), device="cuda"))
    assert y.shape == (0, T, 24) and last.shape == (0, 3, 24)
