"""The group example end to end: what rounds of drafts and verify steps leave of several samples of one prompt is what one
reading of a sample's text leaves."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")


@pytest.mark.parametrize("pool", ["bf16", "e4m3"])
@pytest.mark.parametrize("samples,prompt", [(5, 300), (1, 300), (3, 7)])      # shared pages; a group of one; nothing shared
def test_rounds_leave_what_one_reading_leaves(pool, samples, prompt):
    from examples.verify_group import generate
    r = generate(pool, samples=samples, prompt_len=prompt, rounds=8)
    assert 1 <= r["per_round"] <= 3
    # Both states are made of the attention's outputs, through products of other shapes: a few bf16 roundings (2^-8 each) a
    # token, and in 8 bits a code's step (2^-3) where such a rounding crosses a border, in few places.
    for name in ("rec", "conv"):
        left, read = (t.float() for t in r[name])
        assert (left - read).norm() <= (2.0 ** -5 if pool == "bf16" else 2.0 ** -4) * read.norm(), name
