"""The oracle of the hybrid mixers against independent statements of the same mathematics."""
import numpy as np
import pytest
import torch

from oracle import forward as of
from oracle import hybrid as oh


@pytest.mark.parametrize("width", [2, 3, 4, 8])
def test_conv_is_torchs_depthwise_convolution(width):
    rng = np.random.default_rng(width)
    B, T, C = 2, 11, 5
    x, w, b = rng.standard_normal((B, T, C)), rng.standard_normal((width, C)), rng.standard_normal(C)
    first = rng.standard_normal((B, width - 1, C))
    y, last, states, v, size = oh.conv(x, w, b, first, [T, T], True)
    whole = torch.from_numpy(np.concatenate([first, x], 1)).transpose(1, 2)
    want = torch.nn.functional.conv1d(whole, torch.from_numpy(w.T[:, None].copy()), torch.from_numpy(b), groups=C)
    assert np.abs(torch.nn.functional.silu(want).transpose(1, 2).numpy() - y).max() < 1e-12
    assert np.array_equal(last, np.concatenate([first, x], 1)[:, -(width - 1):]) and np.array_equal(states[:, -1], last)
    assert (size + 1e-12 >= np.abs(v)).all()


def test_conv_in_pieces_and_short_rows():
    rng = np.random.default_rng(1)
    x, w, first = rng.standard_normal((3, 9, 4)), rng.standard_normal((4, 4)), rng.standard_normal((3, 3, 4))
    y, last, states, _, _ = oh.conv(x, w, None, first, [9, 2, 0], False)
    y1, mid, _, _, _ = oh.conv(x[:, :2], w, None, first, [2, 2, 0], False)
    y2, end, _, _, _ = oh.conv(x[:1, 2:], w, None, mid[:1], [7], False)
    assert np.array_equal(np.concatenate([y1[:1], y2], 1), y[:1]) and np.array_equal(end[0], last[0])
    assert np.array_equal(last[2], first[2]) and not y[2].any() and not y[1, 2:].any() and not states[1, 2:].any()
    assert np.array_equal(last[1], [first[1, 2], x[1, 0], x[1, 1]])


def test_scan_closed_form():
    """Constant steps: h_t = sum_s exp(delta a (t - s)) delta b x_s."""
    rng = np.random.default_rng(2)
    T, D, N = 12, 3, 8
    x, a = rng.standard_normal((1, T, D)), -rng.random((D, N))
    b, c = rng.standard_normal((1, 1, 1, N)).repeat(T, 1), rng.standard_normal((1, T, 1, N))
    y, last, states, _ = oh.scan(x, np.full((1, T, D), 0.3), a, b, c, None, None, None, np.zeros((1, D, N)), [T], False)
    for t in range(T):
        h = sum(np.exp(0.3 * a * (t - s)) * 0.3 * x[0, s][:, None] * b[0, 0] for s in range(t + 1))
        assert np.allclose(h, states[0, t], rtol=1e-12) and np.allclose((h * c[0, t]).sum(1), y[0, t], rtol=1e-10)
    assert np.array_equal(last[0], states[0, -1])


def test_scan_groups_gate_softplus_and_lengths():
    rng = np.random.default_rng(3)
    B, T, D, N = 2, 6, 4, 8
    x, dt, z = (rng.standard_normal((B, T, D)) for _ in range(3))
    a, skip, bias = -rng.random((D, N)), rng.standard_normal(D), rng.standard_normal(D)
    b, c = rng.standard_normal((B, T, 2, N)), rng.standard_normal((B, T, 2, N))
    first = rng.standard_normal((B, D, N))
    y, last, _, err = oh.scan(x, dt, a, b, c, skip, z, bias, first, [6, 4], True)
    for g in range(2):      # a group is a scan of its own channels
        s = slice(2 * g, 2 * g + 2)
        step = torch.nn.functional.softplus(torch.from_numpy(dt[..., s] + bias[s])).numpy()
        yg, lg, _, _ = oh.scan(x[..., s], step, a[s], b[:, :, g:g + 1], c[:, :, g:g + 1], skip[s], None, None, first[:, s], [6, 4], False)
        gate = torch.nn.functional.silu(torch.from_numpy(z[..., s])).numpy()
        inside = np.arange(T)[None, :, None] < np.array([6, 4])[:, None, None]
        assert np.allclose(y[..., s], np.where(inside, yg * gate, 0), rtol=1e-10) and np.allclose(last[:, s], lg, rtol=1e-10)
    # the recurrence with one state a channel is the framework's gated recurrence
    g = dt[..., None] * a[:, 0][:, None]
    yr, lr = of.recur(g[..., 0], (dt * x) * b[:, :, :1, 0], first[..., 0], [6, 4])
    _, l1, s1, _ = oh.scan(x, dt, a[:, :1], b[:, :, :1, :1], c[:, :, :1, :1], None, None, None, first[..., :1], [6, 4], False)
    assert np.allclose(s1[..., 0], yr) and np.allclose(l1[..., 0], lr)
    assert all((e >= 0).all() for e in err)


def test_shared_positions():
    table = np.array([[0, 1, 2], [-1, 3, 4], [5, 6, 7], [8, 9, 11]])
    cu, kv = np.array([0, 1, 2, 3, 3]), np.array([300, 200, 300, 300])
    same = lambda rows, n: oh.shared_positions(table, rows, n, cu, kv, 11, 128)
    own = same([0], [])
    assert own[0, 130] == 130 and own[1, 5] == -1 and own[2, 300] == 7 * 128 + 44 and (own[3, 256:] == -1).all()
    got = same([0, 2], [300])                                   # row 1's own token is at 199: one tile
    assert np.array_equal(got[1, :128], own[0, :128]) and np.array_equal(got[1, 128:], own[1, 128:])
    assert np.array_equal(np.delete(got, 1, 0), np.delete(own, 1, 0))
    for rows in ([2, 4], [3, 1], [0, 5], [-1, 2]):              # one row with tokens; no order; out of range
        assert np.array_equal(same(rows, [300]), own)
    assert np.array_equal(same([0, 3], [127]), own) and np.array_equal(same([0, 3], [-5]), own)


def test_pages_of_one_position_are_the_same_cache():
    rng = np.random.default_rng(5)
    k, v, q = rng.standard_normal((4, 2, 6, 8)), rng.standard_normal((4, 2, 6, 8)), rng.standard_normal((3, 4, 8))
    cu, kv, table = np.array([0, 1, 3]), np.array([9, 14]), np.array([[2, 0, -1], [3, 1, 9]])
    a = of.attend(q, cu, kv, table, k, v, 0.3)
    at = oh.shared_positions(table, [0], [], cu, kv, 4, 6)
    b = of.attend(q, cu, kv, at, oh.one_a_page(k), oh.one_a_page(v), 0.3)
    assert all(np.array_equal(x, y) for x, y in zip(a, b)) and a[2].tolist() == [0, of.F_BAD_IDX]
