"""Pins of the forward oracle: torch's e4m3 conversion, a dense softmax, gradients by differences."""
import numpy as np
import pytest
import torch

from oracle import forward as of


def test_e4m3_values_and_rounding_match_torch():
    codes = np.array([c for c in range(256) if c & 0x7F != 0x7F], np.uint8)
    assert np.array_equal(of.e4m3_value(codes), torch.from_numpy(codes).view(torch.float8_e4m3fn).double().numpy())
    rng = np.random.default_rng(0)
    x = rng.standard_normal((64, 128)).astype(np.float32)
    x[1, :8] = [448, 464, 1.0625, 1.1875, 0.001, -0.0009765625, 0, -448]   # ties and sub-normals under s = 0
    x[1, 8:] = 0
    x[2] *= 2.0 ** -140                        # the smallest scale
    x[3] = 0
    code, e, bad = of.quantise(x)
    assert not bad.any() and e[1] == 128 and e[3] == 1 and e[2] == 1
    ref = torch.from_numpy(np.ldexp(x.astype(np.float64), 127 - e.astype(np.int64)[:, None])).float()
    assert np.array_equal(code, ref.to(torch.float8_e4m3fn).view(torch.uint8).numpy())
    amax = np.abs(x.astype(np.float64)).max(-1)
    s = e.astype(np.float64) - 127
    assert np.all(amax <= 448 * 2.0 ** s) and np.all((amax > 448 * 2.0 ** (s - 1)) | (e == 1))
    # half a step of the format at most, and half a sub-normal step below
    off = np.abs(of.cache_values(code, e) - x)
    assert np.all(off <= np.maximum(np.abs(x) * 2.0 ** -4, 2.0 ** (s - 10)[:, None]))


def test_quantise_marks_what_is_not_finite():
    x = np.ones((3, 64))
    x[0, 5], x[1, 6] = np.inf, np.nan
    code, e, bad = of.quantise(x)
    assert list(bad) == [True, True, False] and list(e[:2]) == [255, 255] and not code[:2].any()
    assert np.isnan(of.cache_values(code, e)[:2]).all() and np.array_equal(of.cache_values(code, e)[2], x[2])


def test_attend_matches_a_dense_masked_softmax():
    rng = np.random.default_rng(1)
    B, heads, group, D, ps, pages = 3, 2, 3, 64, 5, 12
    cu, kv = np.array([0, 2, 2, 6], np.int32), np.array([7, 4, 13], np.int32)
    table = rng.permutation(pages).reshape(B, 4).astype(np.int32)
    k, v = rng.standard_normal((2, pages, heads, ps, D))
    q = rng.standard_normal((6, heads * group, D))
    out, lse, flags, _ = of.attend(q, cu, kv, table, k, v, 0.2)
    assert not flags.any()
    for r, t, p, _, _ in of.places(cu, kv, table, pages, ps):
        for h in range(heads * group):
            kk = torch.from_numpy(np.concatenate([k[i, h // group] for i in table[r]])[: p + 1])
            vv = torch.from_numpy(np.concatenate([v[i, h // group] for i in table[r]])[: p + 1])
            s = kk @ torch.from_numpy(q[t, h]) * 0.2
            assert np.allclose(out[t, h], (torch.softmax(s, 0) @ vv).numpy(), atol=1e-13)
            assert np.isclose(lse[t, h], torch.logsumexp(s, 0).item(), atol=1e-13)


def test_attend_rows_that_see_nothing():
    q = np.ones((3, 2, 64))
    k = np.ones((1, 2, 4, 64))
    out, lse, flags, _ = of.attend(q, np.array([0, 2, 3]), np.array([1, 0]), np.array([[0], [0]]), k, k, 1.0)
    assert not out[0].any() and np.isneginf(lse[0]).all() and np.allclose(out[1], 1) and np.isneginf(lse[2]).all()
    out, lse, flags, _ = of.attend(q[:1], np.array([0, 1]), np.array([3]), np.array([[7]]), k, k, 1.0)
    assert flags[0] == of.F_BAD_IDX and not out.any() and np.isneginf(lse).all()


@pytest.mark.parametrize("seed", [0, 1])
def test_recurrence_gradients_by_differences(seed):
    rng = np.random.default_rng(seed)
    B, T, D = 3, 7, 4
    lens = np.array([7, 0, 4])
    g, x = -np.exp(rng.standard_normal((B, T, D))), rng.standard_normal((B, T, D))
    first, dh, d_last = rng.standard_normal((B, D)), rng.standard_normal((B, T, D)), rng.standard_normal((B, D))
    for r in range(B):
        dh[r, lens[r]:] = 0

    def loss(g, x, first):
        h, last = of.recur(g, x, first, lens)
        return (h * dh).sum() + (last * d_last).sum()

    h, _ = of.recur(g, x, first, lens)
    got = of.recur_backward(g, h, dh, first, lens, d_last)
    for i, (grad, at) in enumerate(zip(got, (0, 1, 2))):
        args = [g, x, first]
        for j in np.ndindex(args[at].shape):
            eps = 1e-6
            up, down = [a.copy() for a in args], [a.copy() for a in args]
            up[at][j] += eps
            down[at][j] -= eps
            assert abs((loss(*up) - loss(*down)) / (2 * eps) - grad[j]) < 1e-7


def test_recurrence_forgets_at_minus_infinity():
    g, x = np.zeros((1, 3, 2)), np.ones((1, 3, 2))
    g[0, 1, 0] = -np.inf
    h, last = of.recur(g, x, np.full((1, 2), 5.0), [3])
    assert np.array_equal(h[0, :, 0], [6, 1, 2]) and np.array_equal(last[0], [2, 8])
