"""GPU parity of the paged cache, the attention over it and the recurrence with the float64 oracle.

Tolerances count roundings: half a step of bf16 is 2^-8 relative, of float32 2^-24.
"""
import numpy as np
import pytest
import torch

from oracle import forward as of

pytestmark = pytest.mark.gpu

BF16, F32 = 2.0 ** -8, 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def host(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


class Batch:
    """A paged cache of random contents with `new` tokens of rows of `total` cached ones."""

    def __init__(self, new, total, heads=2, dim=64, page=16, pool="bf16", seed=0, garbage=None, spare=2, interleave=False):
        rng = np.random.default_rng(seed)
        self.rng, self.page, self.pool, self.heads, self.dim = rng, page, pool, heads, dim
        need = [max(0, -(-t // page)) for t in total]
        self.pages = sum(need) + spare
        order = rng.permutation(self.pages)
        self.table = np.full((len(new), max(need + [1])), -1, np.int32)
        at = 0
        for r, m in enumerate(need):
            self.table[r, :m] = order[at:at + m]
            at += m
        self.cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        self.kv_len = np.array(total, np.int32)
        self.N = int(self.cu[-1])
        held = np.zeros((self.pages, page), bool)
        for r, t in enumerate(total):
            for p in range(t):
                held[self.table[r, p // page], p % page] = True
        self.held = held
        x = torch.from_numpy(rng.standard_normal((2, self.pages, heads, page, dim))).to(torch.bfloat16)
        if garbage is not None:
            x[:, torch.from_numpy(~held)[:, None, :].expand(-1, heads, -1)] = garbage
        self.exps = None
        if pool == "e4m3":
            codes, exps, _ = of.quantise(x.double().numpy())
            self.values = of.cache_values(codes, exps)
            kv, self.exps = torch.from_numpy(codes).cuda().view(torch.float8_e4m3fn), torch.from_numpy(exps).cuda()
        else:
            self.values, kv = x.double().numpy(), x.cuda()
        if interleave:      # keys and values of a page side by side in one pool
            kv = kv.view(torch.uint8).transpose(0, 1).contiguous().view(kv.dtype).transpose(0, 1)
            if self.exps is not None:
                self.exps = self.exps.transpose(0, 1).contiguous().transpose(0, 1)
        self.k, self.v = kv[0], kv[1]

    def args(self):
        e = (None, None) if self.exps is None else (self.exps[0], self.exps[1])
        return (dev(self.cu), dev(self.kv_len), dev(self.table), self.k, self.v) + e

    def places(self):
        return of.places(self.cu, self.kv_len, self.table, self.pages, self.page)


# ---------------------------------------------------------------------- cache

CACHES = [
    dict(new=[3], total=[3], page=16),
    dict(new=[1, 0, 5, 2], total=[40, 7, 5, 33], page=16, heads=3),
    dict(new=[3] * 70, total=[5 + r for r in range(70)], page=8, heads=8, dim=128),
    dict(new=[700, 1, 333], total=[700, 90, 600], page=24, heads=5, dim=128),
    dict(new=[17, 4], total=[20, 9], page=1, heads=1),
    dict(new=[2000, 900], total=[2300, 900], page=128, heads=8, dim=128),
]


@pytest.mark.parametrize("case", CACHES)
@pytest.mark.parametrize("pool", ["bf16", "e4m3"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("interleave", [False, True])
def test_cache_write_and_read(case, pool, dtype, interleave):
    from speculative_decoding_verify_07_gb300 import binding as sv
    b = Batch(**case, pool=pool, seed=3, interleave=interleave)
    size = np.exp(2 * b.rng.standard_normal((2, b.N, b.heads, 1)))
    x = torch.from_numpy(b.rng.standard_normal((2, b.N, b.heads, b.dim)) * size).to(dtype)
    x[0, 0, 0] = 0
    # tokens strided, as slices of a fused projection
    wide = torch.zeros((2, b.N, b.heads + 2, b.dim), dtype=dtype)
    wide[:, :, 1:-1] = x
    wide = wide.cuda()
    flags = torch.zeros(len(b.kv_len), dtype=torch.int32, device="cuda")
    sv.spec_cache_write(wide[0, :, 1:-1], wide[1, :, 1:-1], *b.args(), flags=flags)
    k, v = sv.spec_cache_read(b.N, *b.args(), flags=flags)
    torch.cuda.synchronize()
    assert not flags.any()
    pools = [p.view(torch.uint8).cpu().numpy() if pool == "e4m3" else host(p) for p in (b.k, b.v)]
    was = b.values
    touched = np.zeros_like(b.held)
    for i, pool_now in enumerate(pools):
        if pool == "e4m3":
            codes, exps, _ = of.quantise(x[i].double().numpy())
            values, e_now = of.cache_values(codes, exps), b.exps[i].cpu().numpy()
        else:
            values = x[i].to(torch.bfloat16).double().numpy()
        for r, t, p, page, slot in b.places():
            touched[page, slot] = True
            if pool == "e4m3":
                assert np.array_equal(pool_now[page, :, slot], codes[t]) and np.array_equal(e_now[page, :, slot], exps[t])
            else:
                assert np.array_equal(pool_now[page, :, slot], values[t])
        assert np.array_equal(host(k if i == 0 else v), values)
        now = of.cache_values(pool_now, e_now) if pool == "e4m3" else pool_now
        still = np.broadcast_to(~touched[:, None, :], now.shape[:3])
        assert np.array_equal(now[still], was[i][still])      # nothing else was written


@pytest.mark.parametrize("pool", ["bf16", "e4m3"])
def test_cache_write_flags_what_has_no_place_or_is_not_finite(pool):
    from speculative_decoding_verify_07_gb300 import binding as sv
    b = Batch([3, 2, 2, 1, 1], [20, 1, 9, 4, 4], page=4, pool=pool)
    b.table[0, 4] = b.pages            # positions 16..19: tokens 17..19 of row 0
    b.table[2, 2] = -7                 # position 8
    x = torch.ones((2, b.N, b.heads, b.dim), dtype=torch.bfloat16)
    x[0, 7, 1, 3] = np.inf             # row 3
    x[1, 8, 0, 0] = np.nan             # row 4
    flags = torch.zeros(5, dtype=torch.int32, device="cuda")
    sv.spec_cache_write(x[0].cuda(), x[1].cuda(), *b.args(), flags=flags)
    again = torch.zeros_like(flags)
    k, v = sv.spec_cache_read(b.N, *b.args(), flags=again)
    torch.cuda.synchronize()
    assert flags.tolist() == [of.F_BAD_IDX, of.F_BAD_IDX, of.F_BAD_IDX, of.F_NAN, of.F_NAN]
    assert again.tolist() == [of.F_BAD_IDX] * 3 + [0, 0]
    k, v = host(k), host(v)
    none = [t for _, t, _, page, _ in b.places() if page < 0]
    assert none == [0, 1, 2, 3, 6] and not k[none].any() and not v[none].any()
    assert np.array_equal(v[7], np.ones((b.heads, b.dim))) and np.array_equal(k[8], np.ones((b.heads, b.dim)))
    if pool == "e4m3":
        assert np.isnan(k[7, 1]).all() and np.isnan(v[8, 0]).all() and (k[7, 0] == 1).all()
    else:
        assert np.isinf(k[7, 1, 3]) and np.isnan(v[8, 0, 0]) and np.isfinite(k[7]).sum() == k[7].size - 1


# ------------------------------------------------------------------ attention

def check_attend(b, group, scale=None, q_size=2.0, flags=None, expect_flags=None, max_tokens=None, workspace=None,
                 stride=False):
    from speculative_decoding_verify_07_gb300 import binding as sv
    hq = b.heads * group
    q = torch.from_numpy(q_size * b.rng.standard_normal((b.N, hq, b.dim))).to(torch.bfloat16)
    qd = q.cuda()
    if stride:
        wide = torch.zeros((b.N, hq + 3, b.dim), dtype=torch.bfloat16, device="cuda")
        wide[:, :hq] = qd
        qd = wide[:, :hq]
    flags = torch.zeros(len(b.kv_len), dtype=torch.int32, device="cuda")
    most = int((b.cu[1:] - b.cu[:-1]).max()) if max_tokens is None else max_tokens
    out, lse = sv.spec_attend(qd, *b.args(), max_tokens=most, scale=scale, flags=flags, workspace=workspace)
    torch.cuda.synchronize()
    sc = b.dim ** -0.5 if scale is None else scale
    ref, rlse, rflags, size = of.attend(q.double().numpy(), b.cu, b.kv_len, b.table, b.values[0], b.values[1], sc)
    got, glse = host(out), host(lse)
    assert np.array_equal(np.isnan(got), np.isnan(ref)) and np.array_equal(got[np.isinf(ref)], ref[np.isinf(ref)])
    # a score sums dim products in float32 and is off by dim 2^-24 of their sizes; the weights, their rounding to
    # bf16 and the sums over positions follow; the result is rounded once more
    with np.errstate(invalid="ignore"):
        k_top = np.abs(np.where(np.isfinite(b.values[0]), b.values[0], 0)).max()
        s_off = (b.dim + 8) * F32 * np.abs(q.double().numpy()).sum(-1) * k_top * abs(sc)
        tol = BF16 * np.abs(ref) + (BF16 + 2 * s_off[..., None] + 2.0 ** -14) * size + 1e-30
        ok = (np.abs(got - ref) <= tol) | ((got == ref) | (np.isnan(got) & np.isnan(ref)))
        assert ok.all(), (np.argwhere(~ok)[:5], got[~ok][:5], ref[~ok][:5], tol[~ok][:5])
        lok = (np.abs(glse - rlse) <= s_off + 1e-5 + 4 * F32 * np.abs(rlse)) | (glse == rlse) | (np.isnan(glse) & np.isnan(rlse))
        assert lok.all(), (np.argwhere(~lok)[:5], glse[~lok][:5], rlse[~lok][:5])
    assert np.array_equal(flags.cpu().numpy().astype(np.uint32), rflags if expect_flags is None else expect_flags)
    return out, lse


SMALL = [
    dict(new=[1], total=[1]),
    dict(new=[1], total=[333]),
    dict(new=[3, 3, 3], total=[3, 65, 130]),
    dict(new=[1, 0, 5, 2], total=[64, 7, 128, 129], page=5),
    dict(new=[17, 1], total=[300, 17], page=1),
    dict(new=[2] * 40, total=[2 + 7 * r for r in range(40)], page=8),
    dict(new=[1, 1], total=[1500, 1], page=32),
]


@pytest.mark.parametrize("case", SMALL)
@pytest.mark.parametrize("pool", ["bf16", "e4m3"])
@pytest.mark.parametrize("heads,group,dim", [(1, 1, 64), (2, 4, 128), (3, 3, 64), (1, 16, 128), (2, 7, 128)])
def test_attend_small(case, pool, heads, group, dim):
    check_attend(Batch(**case, pool=pool, heads=heads, dim=dim, seed=5, garbage=float("nan")), group)


LARGE = [
    dict(new=[128], total=[128]),
    dict(new=[129, 1, 40], total=[500, 300, 40], page=24),
    dict(new=[257], total=[1111], page=64),
    dict(new=[65, 0, 3, 200], total=[65, 900, 700, 333], page=7),
    dict(new=[1], total=[40], heads=1),
]


@pytest.mark.parametrize("case", LARGE)
@pytest.mark.parametrize("pool", ["bf16", "e4m3"])
@pytest.mark.parametrize("group,dim", [(1, 64), (4, 128), (5, 64), (64, 128), (3, 128)])
def test_attend_chunks(case, pool, group, dim):
    case = dict(dict(heads=1 if group > 8 else 2), **case)
    check_attend(Batch(**case, pool=pool, dim=dim, seed=6, garbage=float("inf")), group)


@pytest.mark.parametrize("pool", ["bf16", "e4m3"])
@pytest.mark.parametrize("most", [1, 17, 4096])
def test_attend_any_hint_gives_the_result(pool, most):
    """max_tokens chooses between kernels and limits nothing."""
    b = Batch([150, 2, 1], [150, 400, 90], pool=pool, dim=128, seed=7)
    check_attend(b, 4, max_tokens=most)


@pytest.mark.parametrize("pool", ["bf16", "e4m3"])
@pytest.mark.parametrize("new", [[3, 2, 2], [130, 2, 2]])
def test_attend_empty_rows_and_bad_pages(pool, new):
    # row 1: more new tokens than cached ones, its first sees nothing; row 2: an empty cache
    b = Batch(new, [new[0] + 60, 1, 0], page=16, pool=pool, seed=8)
    b.table[0, 1] = -1
    b.table[0, 2] = b.pages + 5
    out, lse = check_attend(b, 4)
    t = int(b.cu[1])
    assert not out[t].any() and torch.isneginf(lse[t]).all() and torch.isneginf(lse[t + 2:]).all()
    # a row with no valid page at all
    b.table[0] = -1
    check_attend(b, 4)


@pytest.mark.parametrize("pool", ["bf16", "e4m3"])
@pytest.mark.parametrize("new", [5, 140])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("which", [0, 1])
def test_attend_what_is_not_seen_does_not_arrive(pool, new, bad, which):
    """A key or value that is not finite reaches the tokens at and after its own, none before."""
    b = Batch([new], [new + 70], page=16, pool=pool, heads=1, dim=64, seed=9)
    j = 70 + new // 2
    page, slot = b.table[0, j // 16], j % 16
    if pool == "e4m3":
        b.exps[which, page, 0, slot] = 255
        b.values[which][page, 0, slot] = np.nan
    else:
        (b.k, b.v)[which][page, 0, slot, 3] = bad
        b.values[which][page, 0, slot, 3] = bad
    out, _ = check_attend(b, 2)
    assert torch.isfinite(out[: new // 2]).all()
    if pool == "e4m3" or which == 1 or bad != bad:
        assert not torch.isfinite(out[new // 2:]).all(-1).any()


def test_attend_sizes_of_scores():
    for pool in ("bf16", "e4m3"):
        b = Batch([4, 200], [300, 260], pool=pool, dim=128, seed=10)
        check_attend(b, 4, q_size=60.0)           # weight on one position
        check_attend(b, 4, scale=0.0)             # a plain mean
        check_attend(b, 4, scale=-0.3, stride=True)


def test_attend_strided_pools_share_a_workspace():
    from speculative_decoding_verify_07_gb300 import binding as sv
    ws = sv.new_attend_workspace(2, 4, 128, "cuda")
    for pool in ("bf16", "e4m3"):
        for new, total in (([3] * 9, [700 + 90 * r for r in range(9)]), ([300], [700]), ([1], [9]), ([2, 90], [4000, 90])):
            check_attend(Batch(new, total, pool=pool, dim=128, seed=11, interleave=True), 4, workspace=ws)


def test_attend_graph_replay_and_repeats_are_the_same_bits():
    from speculative_decoding_verify_07_gb300 import binding as sv
    for new, total in (([3] * 20, [50 + 211 * r for r in range(20)]), ([300, 20], [3000, 700])):
        b = Batch(new, total, heads=2, dim=128, pool="e4m3", seed=12)
        q = torch.randn((b.N, 8, 128), device="cuda", dtype=torch.bfloat16)
        ws, args = sv.new_attend_workspace(2, 4, 128, "cuda"), b.args()
        first = [t.clone() for t in sv.spec_attend(q, *args, max_tokens=max(new), workspace=ws)]
        out, lse = torch.empty_like(first[0]), torch.empty_like(first[1])
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            sv.spec_attend(q, *args, max_tokens=max(new), workspace=ws, out=out, lse=lse)
        for _ in range(5):
            out.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, first[0]) and torch.equal(lse, first[1])


def test_attend_on_another_stream():
    from speculative_decoding_verify_07_gb300 import binding as sv
    b = Batch([3, 3], [900, 70], dim=128, seed=13)
    q = torch.randn((6, 8, 128), device="cuda", dtype=torch.bfloat16)
    args = b.args()
    want = sv.spec_attend(q, *args, max_tokens=3)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = sv.spec_attend(q, *args, max_tokens=3, stream=side)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_cache_offsets_past_32_bits():
    """Pages whose byte offsets pass 2^32, and whose element offsets pass 2^31."""
    from speculative_decoding_verify_07_gb300 import binding as sv
    pages, heads, ps, D = 36000, 8, 64, 128
    k = torch.empty((pages, heads, ps, D), dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    table = torch.tensor([[0, 33000, 35999]], dtype=torch.int32, device="cuda")
    n = 3 * ps - 5
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    kv = torch.tensor([n], dtype=torch.int32, device="cuda")
    x = torch.randn((2, n, heads, D), device="cuda").to(torch.bfloat16)
    sv.spec_cache_write(x[0], x[1], cu, kv, table, k, v)
    rk, rv = sv.spec_cache_read(n, cu, kv, table, k, v)
    assert torch.equal(rk, x[0]) and torch.equal(rv, x[1])
    assert torch.equal(k[35999, :, 3], x[0, 2 * ps + 3])
    q = torch.randn((n, heads, D), device="cuda").to(torch.bfloat16)
    for last in (1, n):
        cu2 = torch.tensor([0, last], dtype=torch.int32, device="cuda")
        out, _ = sv.spec_attend(q[n - last:], cu2, kv, table, k, v, max_tokens=last)
        s = torch.einsum("nhd,mhd->hnm", q[n - last:].double(), x[0].double()) * D ** -0.5
        seen = torch.arange(n, device="cuda")[None] <= torch.arange(n - last, n, device="cuda")[:, None]
        w = torch.softmax(s.masked_fill(~seen, -torch.inf), -1)
        ref = torch.einsum("hnm,mhd->nhd", w, x[1].double())
        size = torch.einsum("hnm,mhd->nhd", w, x[1].double().abs())
        assert ((out.double() - ref).abs() <= BF16 * ref.abs() + 1.05 * BF16 * size).all()


# ----------------------------------------------------------------- recurrence

def run_recur(B, T, D, dtype, h_dtype, seed=0, state=True, lens=None, slots=None, stride=False, resets=0.0, memory=4.0,
              workspace=None):
    from speculative_decoding_verify_07_gb300 import binding as sv
    rng = np.random.default_rng(seed)
    g = -np.exp(rng.uniform(-memory, 0.0, D) + 0.5 * rng.standard_normal((B, T, D)))
    if resets:
        g[rng.random((B, T)) < resets] = -np.inf
    g = torch.from_numpy(g).to(dtype)
    x = torch.from_numpy(rng.standard_normal((B, T, D))).to(dtype)
    dh = torch.from_numpy(rng.standard_normal((B, T, D))).to(dtype)
    d_last = rng.standard_normal((B, D)).astype(np.float32)
    slot = rng.permutation(B + 3)[:B].astype(np.int32) if state else None
    st = rng.standard_normal((B + 3, D)).astype(np.float32) if state else None
    ln = np.full(B, T) if lens is None else np.array(lens)
    gd, xd = g.cuda(), x.cuda()
    if stride:       # two halves of one projection, padded rows
        both = torch.full((B, T + 1, 2 * D), float("nan"), dtype=dtype, device="cuda")
        both[:, :T, :D], both[:, :T, D:] = gd, xd
        gd, xd = both[:, :T, :D], both[:, :T, D:]
    for r in range(B):      # what lies beyond a row's length is never read
        gd[r, ln[r]:] = float("nan")
        xd[r, ln[r]:] = float("nan")
    sd, sl = (dev(st), dev(slot)) if state else (None, None)
    lend = None if lens is None else dev(ln.astype(np.int32))
    flags = torch.zeros(B, dtype=torch.int32, device="cuda")
    dhd = dh.cuda()
    for r in range(B):
        dhd[r, ln[r]:] = float("nan")
    h, last = sv.spec_recur(gd, xd, sd, sl, lend, h_dtype=h_dtype, flags=flags, workspace=workspace)
    dg, dx, d_state = sv.spec_recur_backward(gd, h, dhd, sd, sl, lend, dev(d_last), flags=flags, workspace=workspace)
    torch.cuda.synchronize()
    assert not flags.any()
    first = st[slot].astype(np.float64) if state else np.zeros((B, D))
    g64, x64, dh64 = g.double().numpy(), x.double().numpy(), dh.double().numpy()
    rh, rlast = of.recur(g64, x64, first, ln)
    rdg, rdx, rds = of.recur_backward(g64, host(h), dh64, first, ln, d_last.astype(np.float64))
    # each step rounds three times (exp within 2 units of 2^-24, the multiply-add, and when the steps are joined a
    # product of decays): errors add over the steps with the same weights as |x|
    steps = 12 * F32 * (1 + np.arange(T)[None, :, None])
    hsize, lsize = of.recur(g64, np.abs(x64), np.abs(first), ln)
    _, dsize, dssize = of.recur_backward(g64, host(h), np.abs(dh64), np.abs(first), ln, np.abs(d_last.astype(np.float64)))
    back = 12 * F32 * (1 + T - np.arange(T)[None, :, None])
    ho, go = (F32 if h_dtype == torch.float32 else BF16), (F32 if dtype == torch.float32 else BF16)

    def near(got, ref, tol, what):
        ok = np.abs(got - ref) <= tol + 1e-37
        assert ok.all(), (what, np.argwhere(~ok)[:5], got[~ok][:5], ref[~ok][:5], tol[~ok][:5])

    near(host(h), rh, ho * np.abs(rh) + steps * hsize, "h")
    near(host(last), rlast, 12 * F32 * (T + 1) * lsize, "last")
    near(host(dx), rdx, go * np.abs(rdx) + back * dsize, "dx")
    hb = np.concatenate([np.abs(first)[:, None], np.abs(host(h))[:, :-1]], 1)
    near(host(dg), rdg, go * np.abs(rdg) + (back + 4 * F32) * dsize * np.exp(g64) * hb, "dg")
    near(host(d_state), rds, 12 * F32 * (T + 1) * dssize, "d_state")
    for r in range(B):
        assert not host(h)[r, ln[r]:].any() and not host(dg)[r, ln[r]:].any() and not host(dx)[r, ln[r]:].any()


DT = [torch.bfloat16, torch.float32]


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("h_dtype", DT)
@pytest.mark.parametrize("B,T,D", [(1, 1, 64), (3, 3, 1), (2, 17, 33), (4, 2, 4096), (2, 100, 130), (1, 511, 64),
                                   (2, 512, 96), (1, 513, 65), (2, 2500, 70)])
def test_recur(B, T, D, dtype, h_dtype):
    run_recur(B, T, D, dtype, h_dtype, seed=B + T + D)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("T", [3, 40, 1100])
def test_recur_lengths_strides_and_no_state(dtype, T):
    lens = [T, 0, 1, T // 2, T - 1]
    run_recur(5, T, 72, dtype, dtype, seed=1, lens=lens)
    run_recur(5, T, 72, dtype, torch.float32, seed=2, lens=lens, stride=True, state=False)
    run_recur(5, T, 71, dtype, dtype, seed=3, stride=True, resets=0.1)


@pytest.mark.parametrize("dtype", DT)
def test_recur_long(dtype):
    run_recur(1, 20000, 40, dtype, torch.float32, seed=4, memory=9.0, resets=1e-4)
    run_recur(2, 9000, 256, dtype, dtype, seed=5, lens=[9000, 4097])


def test_recur_shapes_share_a_workspace():
    from speculative_decoding_verify_07_gb300 import binding as sv
    ws = sv.new_recur_workspace(3, 5000, 200, "cuda")
    for i, (B, T, D) in enumerate([(3, 5000, 200), (2, 3000, 65), (1, 5000, 200), (3, 600, 128), (2, 1, 64), (3, 5000, 199)]):
        run_recur(B, T, D, DT[i % 2], DT[i // 2 % 2], seed=20 + i, workspace=ws)


def test_recur_repeats_and_graph_replays_are_the_same_bits():
    from speculative_decoding_verify_07_gb300 import binding as sv
    B, T, D = 2, 6000, 128
    g = -torch.rand((B, T, D), device="cuda").to(torch.bfloat16)
    x, dh = (torch.randn((B, T, D), device="cuda").to(torch.bfloat16) for _ in range(2))
    ws = sv.new_recur_workspace(B, T, D, "cuda")
    h, last = sv.spec_recur(g, x, workspace=ws)
    want = [h, last, *sv.spec_recur_backward(g, h, dh, workspace=ws)]
    got = [torch.empty_like(t) for t in want]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sv.spec_recur(g, x, h=got[0], last=got[1], workspace=ws)
        sv.spec_recur_backward(g, got[0], dh, dg=got[2], dx=got[3], d_state=got[4], workspace=ws)
    for _ in range(5):
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_recur_steps_in_place_continue_a_scan():
    """A prompt, then single steps on the cached state, against one long scan."""
    from speculative_decoding_verify_07_gb300 import binding as sv
    B, T, D = 4, 90, 256
    g = -torch.rand((B, T, D), device="cuda")
    x = torch.randn((B, T, D), device="cuda")
    whole, _ = sv.spec_recur(g, x)
    cache, slot = torch.zeros((6, D), device="cuda"), torch.tensor([5, 0, 3, 1], dtype=torch.int32, device="cuda")
    got = [sv.spec_recur(g[:, :70], x[:, :70], cache, slot, last=cache, last_slot=slot)[0]]
    for t in range(70, T):
        got.append(sv.spec_recur(g[:, t:t + 1], x[:, t:t + 1], cache, slot, last=cache, last_slot=slot)[0])
    got = torch.cat(got, 1)
    assert (got - whole).abs().max() <= 12 * F32 * T * whole.abs().max()
    assert torch.equal(cache[slot.long()], got[:, -1]) and not cache[[2, 4]].any()


def test_recur_bad_slots_are_flagged_and_left_alone():
    from speculative_decoding_verify_07_gb300 import binding as sv
    for T in (3, 1500):
        B, D = 3, 64
        g, x = torch.zeros((B, T, D), device="cuda"), torch.ones((B, T, D), device="cuda")
        state = torch.ones((4, D), device="cuda")
        slot = torch.tensor([0, 4, -1], dtype=torch.int32, device="cuda")
        flags = torch.zeros(B, dtype=torch.int32, device="cuda")
        last = torch.full((B, D), 7.0, device="cuda")
        h, _ = sv.spec_recur(g, x, state, slot, last=last, flags=flags)
        assert flags.tolist() == [0, of.F_BAD_IDX, of.F_BAD_IDX]
        assert torch.equal(h[0, :, 0], 2 + torch.arange(T, device="cuda").float()) and not h[1:].any()
        assert (last[0] == T + 1).all() and (last[1:] == 7).all()
        flags.zero_()
        dg, dx, ds = sv.spec_recur_backward(g, h, x, state, slot, flags=flags)
        assert flags.tolist() == [0, of.F_BAD_IDX, of.F_BAD_IDX]
        assert (ds[0] == T).all() and not dg[1:].any() and not dx[1:].any() and not ds[1:].any()


def test_recur_states_commit():
    """The scan's states are one layer of spec_commit's verify buffer."""
    from speculative_decoding_verify_07_gb300 import binding as sv
    L, B, S, D, slots = 2, 5, 3, 96, 7
    cache = torch.randn((L, slots, 1, 1, D), device="cuda")
    slot = torch.tensor([6, 2, 0, 1, 4], dtype=torch.int32, device="cuda")
    g = -torch.rand((L, B, S, D), device="cuda").to(torch.bfloat16)
    x = torch.randn((L, B, S, D), device="cuda").to(torch.bfloat16)
    verify = torch.empty((L, B, S, 1, 1, D), device="cuda")
    for l in range(L):
        sv.spec_recur(g[l], x[l], cache[l].view(slots, D), slot, h=verify[l].view(B, S, D))
    accept = torch.tensor([1, 2, 3, 0, 2], dtype=torch.int32, device="cuda")
    was = cache.clone()
    sv.spec_commit(verify, None, accept, slot, cache, None)
    for l in range(L):
        for r in range(B):
            a = int(accept[r])
            want = sv.spec_recur(g[l, r:r + 1, :a], x[l, r:r + 1, :a], was[l].view(slots, D), slot[r:r + 1])[1][0] if a \
                else was[l, slot[r], 0, 0]
            assert torch.equal(cache[l, slot[r], 0, 0], want)
