"""Edges of the causal convolution, the selective scan and the attention over a shared prefix on the GPU.

Tolerances count roundings: half a step of bf16 is 2^-8 relative, of float32 2^-24.
"""
import numpy as np
import pytest
import torch

from oracle import forward as of
from oracle import hybrid as oh
from tests.test_gpu_forward import Batch
from tests.test_gpu_hybrid import DT, F32, half, host, near, run_scan
from tests.test_gpu_shared import check, share

pytestmark = pytest.mark.gpu


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


# ------------------------------------------------------------------- the scan

@pytest.mark.parametrize("B,T,D,N,groups", [(8, 2048, 512, 8, 8), (9, 8192, 64, 16, 2), (5, 1279, 384, 32, 8), (7, 2934, 312, 16, 2),
                                            (2, 1551, 1338, 16, 2), (1, 2048, 1728, 16, 36)])
def test_scan_stays_within_its_workspace(B, T, D, N, groups):
    """Several groups that divide a row otherwise than one: what lies behind a workspace of the size asked for is untouched."""
    from speculative_decoding_verify_07_gb300 import binding as sv
    size = sv.LIB.spec_scan_workspace_size(B, T, D, N)
    whole = torch.full((size + (8 << 20),), 0xa5, dtype=torch.uint8, device="cuda")
    run_scan(B, T, D, N, torch.bfloat16, groups=groups, seed=B + T, workspace=whole[:size])
    assert (whole[size:] == 0xa5).all()


def test_scan_workspace_serves_smaller_batches():
    from speculative_decoding_verify_07_gb300 import binding as sv
    ws = sv.new_scan_workspace(8, 3000, 2048, 16, "cuda")
    for B, T in ((8, 50), (1, 3000), (3, 1000)):
        run_scan(B, T, 2048, 16, torch.bfloat16, seed=T, workspace=ws)


@pytest.mark.parametrize("T", [1, 17])
def test_scan_steps_far_below_zero(T):
    """softplus on both sides of where exp(v) leaves the normal numbers: as exact as elsewhere above, zero below, and a token
    of such a step leaves the state to the bit."""
    from speculative_decoding_verify_07_gb300 import binding as sv
    above, below = np.linspace(-87.33, -80.0, 500), np.array([-87.34, -87.5, -88.0, -88.8, -95.0, -104.0, -1e4, -3e38, -np.inf])
    v = torch.from_numpy(np.concatenate([above, below]).astype(np.float32))
    D, N = v.numel(), 8
    x, b = torch.ones((1, T, D), device="cuda"), torch.ones((1, T, 1, N), device="cuda")
    a = torch.full((D, N), -1.0, device="cuda")
    dt = torch.full((1, T, D), -float("inf"))
    dt[0, T // 2] = v
    _, last = sv.spec_scan(x, dt.cuda(), a, b, b)
    want = np.exp(v.double().numpy())[:500]          # (ln(1 + e) is e there)
    near(host(last)[0, :500, 0], want, 13 * F32 * want - 1e-37, "softplus")
    assert not last[0, 500:].any()
    state = torch.randn((1, D, N), device="cuda")
    dt[0, T // 2] = -float("inf")
    _, last = sv.spec_scan(x, dt.cuda(), a, b, b, None, None, None, state)
    assert torch.equal(last, state)


@pytest.mark.parametrize("T", [3, 16, 33, 1000])
def test_scan_states_that_are_forgotten_at_once(T):
    """a of -inf and of the lowest numbers: a state is what the last token puts in, whatever the row's length, and a row
    without tokens keeps what it had."""
    from speculative_decoding_verify_07_gb300 import binding as sv
    D, N, lens = 24, 8, [T, T // 2 + 1, 1, 0]
    x, b, c = (torch.randn(s, device="cuda") for s in ((4, T, D), (4, T, 1, N), (4, T, 1, N)))
    dt = torch.rand((4, T, D), device="cuda") + 0.01
    state = torch.randn((4, D, N), device="cuda")
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    a = -torch.rand((D, N), device="cuda")
    got = []
    for low in (-2e38, -3.4e38, -float("inf")):
        a[1::2, 3] = low
        got.append(sv.spec_scan(x, dt, a, b, c, None, None, None, state, None, n, softplus=False))
    for y, last in got:
        assert torch.isfinite(y).all() and torch.equal(y, got[0][0]) and torch.equal(last, got[0][1])
        for r, m in enumerate(lens):
            want = host(dt[r, m - 1, 1::2]) * host(x[r, m - 1, 1::2]) * host(b[r, m - 1, 0, 3]) if m else host(state[r, 1::2, 3])
            near(host(last[r, 1::2, 3]), want, 2.1 * F32 * np.abs(want), "last")


def infinite_scan(T, edit):
    """A scan of fast states (decays of a token from exp(-0.1) to exp(-16), none of more than a few tokens above 2^-126) with
    something infinite put in by `edit`, against the oracle: the same infinities and NaN, and all else as ever."""
    from speculative_decoding_verify_07_gb300 import binding as sv
    rng = np.random.default_rng(T)
    B, D, N = 2, 24, 16
    x, b, c = (rng.standard_normal(s).astype(np.float32) for s in ((B, T, D), (B, T, 1, N), (B, T, 1, N)))
    dt = rng.uniform(0.1, 1.0, (B, T, D)).astype(np.float32)
    a = np.tile(-np.arange(1.0, N + 1), (D, 1)).astype(np.float32)
    state = rng.standard_normal((B, D, N)).astype(np.float32)
    edit(x, b, state)
    move = lambda v: torch.from_numpy(v).cuda()
    y, last = sv.spec_scan(move(x), move(dt), move(a), move(b), move(c), None, None, None, move(state), softplus=False)
    with np.errstate(all="ignore"):
        wy, wl, _, (ey, el, _) = oh.scan(x, dt, a, b, c, None, None, None, state, [T] * B, False)
    for got, want, err in ((host(y), wy, F32 * ey + F32 * np.abs(wy)), (host(last), wl, F32 * el)):
        assert np.array_equal(np.isnan(got), np.isnan(want)) and np.array_equal(got[np.isinf(want)], want[np.isinf(want)])
        there = np.isfinite(want)
        near(got[there], want[there], err[there], "finite")
    return wl


@pytest.mark.parametrize("T", [3, 40, 300, 1500])
def test_scan_infinite_states_stay(T):
    def edit(x, b, state):
        state[0, 3] = np.inf
        state[0, 4, ::2] = -np.inf
        state[1, 23, 15] = np.inf
    wl = infinite_scan(T, edit)
    assert np.isinf(wl[0, 3]).all() and np.isinf(wl[1, 23, 15])


@pytest.mark.parametrize("T", [3, 40, 300, 1500])
def test_scan_infinite_inputs_stay(T):
    """Infinities in the first, a middle and the last token; opposite ones cancel to NaN, also against an infinite state."""
    def edit(x, b, state):
        x[0, 0, 3] = np.inf
        x[0, T // 2, 5] = -np.inf
        x[0, T - 1, 6] = np.inf
        x[0, 1, 7], x[0, T - 2, 7] = np.inf, -np.inf
        b[1, T // 2, 0, 2] = -np.inf
        state[0, 9], x[0, T // 2, 9] = np.inf, -np.inf
    wl = infinite_scan(T, edit)
    assert np.isinf(wl[0, 3]).all() and np.isinf(wl[1, :, 2]).all() and not np.isfinite(wl[0, 9]).any()


def test_scan_infinite_inputs_leave_the_others_alone():
    """The same bits in all channels and rows that nothing infinite enters."""
    from speculative_decoding_verify_07_gb300 import binding as sv
    B, T, D, N = 2, 2000, 24, 16
    x, dt, b = (torch.randn(s, device="cuda") for s in ((B, T, D), (B, T, D), (B, T, 1, N)))
    a = -torch.rand((D, N), device="cuda")
    want = [t.clone() for t in sv.spec_scan(x, dt, a, b, b)]
    x[0, 700, 5] = float("inf")
    got = sv.spec_scan(x, dt, a, b, b)
    others = torch.tensor([d for d in range(D) if d != 5], device="cuda")
    for g, w, channels in zip(got, want, (1, 0)):
        assert torch.equal(g[1], w[1]) and torch.equal(g[0].index_select(channels, others), w[0].index_select(channels, others))
    assert torch.isinf(got[1][0, 5]).all()


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("D", [24, 26])
def test_scan_infinite_inputs_of_groups_and_ragged_rows(D, dtype):
    from speculative_decoding_verify_07_gb300 import binding as sv
    B, T, N, lens = 3, 1300, 8, [1300, 901, 130]
    gen = torch.Generator().manual_seed(D)
    x, dt = (torch.randn((B, T, D), generator=gen).to(dtype) for _ in range(2))
    b, c = (torch.randn((B, T, 2, N), generator=gen).to(dtype) for _ in range(2))
    a, skip, bias = -torch.arange(1.0, N + 1).repeat(D, 1), torch.randn(D, generator=gen), torch.ones(D)
    x[0, 100, 3], x[0, 700, D - 1], x[1, 880, 5], x[2, 0, 7] = float("inf"), -float("inf"), float("inf"), float("inf")
    b[1, 300, 1, 4] = float("inf")
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    y, last = sv.spec_scan(*(v.cuda() for v in (x, dt, a, b, c, skip)), None, bias.cuda(), lens=n)
    with np.errstate(all="ignore"):
        wy, wl, _, (ey, el, _) = oh.scan(*(host(v) for v in (x, dt, a, b, c, skip)), None, host(bias), np.zeros((B, D, N)), lens, True)
    for got, want, err in ((host(y), wy, half(dtype) * np.abs(wy) + F32 * ey), (host(last), wl, F32 * el)):
        assert np.array_equal(np.isnan(got), np.isnan(want)) and np.array_equal(got[np.isinf(want)], want[np.isinf(want)])
        there = np.isfinite(want)
        near(got[there], want[there], err[there], "finite")
    assert np.isinf(wl[0, 3]).all() and np.isinf(wl[1, D // 2:, 4]).all() and np.isfinite(wl[1, :5]).all()


# -------------------------------------------------------- the shared attention

@pytest.mark.parametrize("group", [1, 40])
def test_more_common_tiles_than_a_call_takes(group):
    """2^31 tiles and more (two rows that see one page again and again): as spec_attend, nothing is written and row 0 flagged;
    the workspace serves on."""
    from speculative_decoding_verify_07_gb300 import binding as sv
    heads, page, most, dim = 140, 4096, 524287, 64
    kv = torch.randn((1, heads, page, dim), device="cuda").to(torch.bfloat16)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
    table = torch.zeros((2, most), dtype=torch.int32, device="cuda")
    q = torch.randn((2, heads * group, dim), device="cuda").to(torch.bfloat16)
    ws = sv.new_attend_shared_workspace(2, 2, heads, group, dim, "cuda")

    def call(kv_len):
        out, lse = torch.full_like(q, 7.0), torch.full(q.shape[:2], 7.0, device="cuda")
        flags = i32(0, 0)
        sv.spec_attend_shared(q, i32(0, 2), i32(0x7fffffff), i32(0, 1, 2), i32(*kv_len), table, kv, kv, max_tokens=1, out=out, lse=lse,
                              flags=flags, workspace=ws)
        return out, lse, flags.tolist()

    want = call((700, 650))
    assert want[2] == [0, 0] and torch.isfinite(want[1]).all() and (want[0] != 7).all()
    out, lse, flags = call((most * page, most * page))
    assert flags == [of.F_BAD_IDX, 0] and (out == 7).all() and (lse == 7).all()
    again = call((700, 650))
    assert again[2] == [0, 0] and torch.equal(again[0], want[0]) and torch.equal(again[1], want[1])


@pytest.mark.parametrize("pool", ["bf16", "e4m3"])
@pytest.mark.parametrize("most", [3, 4096])
def test_more_groups_and_rows_than_a_cta_has_warps_and_threads(most, pool):
    """1040 rows in 90 groups of uneven sizes, some empty, some of one row, rows of no group before and behind them."""
    rng = np.random.default_rng(7)
    new = rng.integers(0, 3, 1040)
    new[[10, 600, 1039]] = 4, 3, 2
    rows = np.sort(rng.integers(7, 1030, 91))
    rows[20] = rows[21] = rows[19]
    lens = rng.integers(0, 420, 90).tolist()
    total = new + rng.integers(100, 240, 1040)
    b = Batch(new.tolist(), total.tolist(), page=32, heads=1, dim=64, pool=pool, seed=21)
    share(b, rows.tolist(), lens)
    check(b, 2, rows.tolist(), lens, max_tokens=most)


# ------------------------------------------------------------------ the ranges

def test_the_longest_rows():
    """SPEC_MAX_LENGTH tokens of one value each (strides of zero), which both operators soon answer alike: offsets, tiles and
    segments count in 64 bits where 32 do not hold them."""
    from speculative_decoding_verify_07_gb300 import binding as sv
    T, N, n = 0x7fffff00, 8, 0x7fffff00 - 1000
    one = torch.ones((1, 1, 1), dtype=torch.bfloat16, device="cuda")
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    w = torch.tensor([[0.5], [0.25], [2.0]], device="cuda")
    y, last = sv.spec_conv(one.expand(1, T, 1), w, lens=lens, silu=False)
    assert y[0, :2, 0].tolist() == [2.0, 2.25] and (y[0, 2:n:1000003] == 2.75).all() and (y[0, n - 3:n] == 2.75).all()
    assert not y[0, n:].any() and (last == 1).all()
    del y
    b = torch.ones((1, 1, 1, N), dtype=torch.bfloat16, device="cuda").expand(1, T, 1, N)
    a = -torch.arange(1, N + 1, device="cuda").float().view(1, N)
    y, last = sv.spec_scan(one.expand(1, T, 1), (0.5 * one).expand(1, T, 1), a, b, b, lens=lens, softplus=False)
    # h = 1/2 (1 + e + e^2 + ...) with e = exp(a / 2), 1 / (1 - e) tokens remembered, each with less than 30 roundings as the
    # oracle counts them
    e = np.exp(-0.5 * np.arange(1, N + 1))
    want = 0.5 / (1 - e)
    near(host(last)[0, 0], want, 30 * F32 * want / (1 - e), "last")
    some = host(torch.cat([y[0, 100:n:1000003, 0], y[0, n - 100:n, 0]]))
    near(some, np.full_like(some, want.sum()), half(torch.bfloat16) * want.sum() + 300 * F32, "y")
    assert not y[0, n:].any()


def test_the_most_rows():
    from speculative_decoding_verify_07_gb300 import binding as sv
    B, C, N = 65535, 9, 8
    x, dt, b = (torch.randn(s, device="cuda") for s in ((B, 1, C), (B, 1, C), (B, 1, 1, N)))
    w, a = torch.randn((3, C), device="cuda"), -torch.rand((C, N), device="cuda")
    y, last = sv.spec_conv(x, w, silu=False)
    assert torch.equal(y[:, 0], x[:, 0] * w[2]) and torch.equal(last[:, 1], x[:, 0]) and not last[:, 0].any()
    y, last = sv.spec_scan(x, dt, a, b, b, softplus=False)
    want = (dt[:, 0] * x[:, 0])[..., None] * b[:, 0]
    assert torch.equal(last, want)
    full = (want.double() * b[:, 0].double()).sum(-1)
    near(host(y)[:, 0], host(full), 2 * N * F32 * host((want * b[:, 0]).abs().sum(-1)), "y")
    with pytest.raises(sv.SpecError):
        sv.spec_conv(torch.zeros((B + 1, 1, 1), device="cuda"), torch.ones((2, 1), device="cuda"))
