"""Edges of the forward oracle: page tables shorter than the rows."""
import numpy as np
import pytest

from oracle import forward as of


@pytest.mark.parametrize("wide", [2, 1, 0])
def test_attend_beyond_the_table(wide):
    rng = np.random.default_rng(0)
    k, v = rng.standard_normal((2, 3, 1, 4, 64))
    table, q = np.array([[2, 0]])[:, :wide], rng.standard_normal((1, 1, 64))
    out, lse, flags, _ = of.attend(q, [0, 1], [11], table, k, v, 0.1)
    assert flags[0] == of.F_BAD_IDX
    if not wide:
        assert not out.any() and np.isneginf(lse).all()
        return
    # what the table reaches, as if the row ended there
    want, wl, none, _ = of.attend(q, [0, 1], [4 * wide], table, k, v, 0.1)
    assert none[0] == 0 and np.array_equal(out, want) and np.array_equal(lse, wl)
