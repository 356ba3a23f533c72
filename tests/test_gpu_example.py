"""The example end to end: serving rounds leave what one reading of the same tokens leaves; the gates learn."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")


@pytest.mark.parametrize("pool", ["bf16", "e4m3"])
def test_rounds_leave_what_a_prompt_leaves(pool):
    from examples.verify_forward import generate
    r = generate(pool, batch=5, rounds=10)
    assert 1 < r["per_round"] <= 3
    # Keys and values of layer one come from the tokens alone, by products of other shapes: bf16 roundings apart, and
    # in 8 bits a code's step (2^-3) where such a rounding crosses a border, in few places.
    left, read = (t.float() for t in r["cache"])
    assert (left - read).norm() <= (2.0 ** -7 if pool == "bf16" else 2.0 ** -5) * read.norm()
    # The states sum outputs of the layer before: a few bf16 roundings a token (2^-8 each), and the cache's.
    left, read = r["states"]
    assert (left - read).norm() <= (2.0 ** -5 if pool == "bf16" else 2.0 ** -4) * read.norm()


def test_gates_learn():
    from examples.verify_forward import fit_gates
    losses = fit_gates()
    assert losses[-1] < 0.05 * losses[0] and all(b == b for b in losses)
