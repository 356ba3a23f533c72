"""GPU parity of the attention over a shared prefix with the float64 oracle, and with spec_attend.

Tolerances as in test_gpu_forward: half a step of bf16 is 2^-8 relative, of float32 2^-24.
"""
import numpy as np
import pytest
import torch

from oracle import forward as of
from oracle import hybrid as oh
from tests.test_gpu_forward import BF16, F32, Batch, dev, host

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")


def share(b, rows, lens):
    """Lets each group's rows find their common whole pages in the first row's; a page begun keeps its own (other) contents."""
    for g, n in enumerate(lens):
        for r in range(rows[g] + 1, rows[g + 1]):
            m = min(n // b.page, b.table.shape[1])
            b.table[r, :m] = b.table[rows[g], :m]


def check(b, group, rows, lens, scale=None, q_size=2.0, max_tokens=None, workspace=None, stride=False):
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
    rd, ld = dev(np.array(rows, np.int32)), dev(np.array(lens, np.int32))
    # (what belongs to no row is left alone)
    out = torch.full((b.N + 2, hq, b.dim), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((b.N + 2, hq), 7.0, device="cuda")
    qx = torch.cat([qd, qd[:2] if b.N > 1 else qd[:1].expand(2, -1, -1)])
    sv.spec_attend_shared(qx, rd, ld, *b.args(), max_tokens=most, scale=scale, out=out, lse=lse, flags=flags, workspace=workspace)
    torch.cuda.synchronize()
    assert (out[b.N:] == 7).all() and (lse[b.N:] == 7).all()
    sc = b.dim ** -0.5 if scale is None else scale
    at = oh.shared_positions(b.table, rows, lens, b.cu, b.kv_len, b.pages, b.page)
    ref, rlse, rflags, size = of.attend(q.double().numpy(), b.cu, b.kv_len, at, oh.one_a_page(b.values[0]), oh.one_a_page(b.values[1]), sc)
    got, glse = host(out[:b.N]), host(lse[:b.N])
    assert np.array_equal(np.isnan(got), np.isnan(ref)) and np.array_equal(got[np.isinf(ref)], ref[np.isinf(ref)])
    with np.errstate(invalid="ignore"):
        k_top = np.abs(np.where(np.isfinite(b.values[0]), b.values[0], 0)).max()
        s_off = (b.dim + 8) * F32 * np.abs(q.double().numpy()).sum(-1) * k_top * abs(sc)
        tol = BF16 * np.abs(ref) + (BF16 + 2 * s_off[..., None] + 2.0 ** -14) * size + 1e-30
        ok = (np.abs(got - ref) <= tol) | ((got == ref) | (np.isnan(got) & np.isnan(ref)))
        assert ok.all(), (np.argwhere(~ok)[:5], got[~ok][:5], ref[~ok][:5], tol[~ok][:5])
        lok = (np.abs(glse - rlse) <= s_off + 1e-5 + 4 * F32 * np.abs(rlse)) | (glse == rlse) | (np.isnan(glse) & np.isnan(rlse))
        assert lok.all(), (np.argwhere(~lok)[:5], glse[~lok][:5], rlse[~lok][:5])
    assert np.array_equal(flags.cpu().numpy().astype(np.uint32), rflags)
    return out[:b.N], lse[:b.N]


CASES = [
    # (new, total, rows, lens, page)
    ([1, 1], [150, 160], [0, 2], [140], 16),
    ([3, 3, 3, 3], [300, 290, 513, 280], [0, 4], [277], 16),
    ([1] * 5, [400, 401, 129, 700, 131], [0, 2, 5], [256, 128], 8),
    ([2, 0, 1, 4, 3, 1], [390, 600, 391, 400, 20, 300], [0, 4], [384], 24),          # an empty row; rows of no group
    ([5, 1], [133, 129], [0, 2], [1000], 1),                                          # shared up to the new tokens
    ([1, 1, 1], [140, 3, 600], [0, 3], [130], 16),                                    # a row too short for any
    ([40, 7, 33], [700, 650, 680], [0, 3], [640], 128),
    ([130, 1, 64], [900, 700, 764], [1, 3], [699], 32),
    ([1] * 64, [260 + 5 * r for r in range(64)], [0, 64], [256], 16),
    ([2] * 24, [520 + 3 * r for r in range(24)], [0, 3, 3, 4, 16, 24], [512, 128, 256, 400, 512], 16),
]


@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("pool", ["bf16", "e4m3"])
@pytest.mark.parametrize("heads,group,dim", [(1, 1, 64), (2, 4, 128), (3, 3, 64), (1, 16, 128)])
def test_shared(case, pool, heads, group, dim):
    new, total, rows, lens, page = case
    b = Batch(new, total, page=page, pool=pool, heads=heads, dim=dim, seed=7, garbage=float("nan"))
    share(b, rows, lens)
    check(b, group, rows, lens)


@pytest.mark.parametrize("pool", ["bf16", "e4m3"])
def test_shared_long(pool):
    new, total = [3] * 12, [9000 + 37 * r for r in range(12)]
    b = Batch(new, total, page=64, pool=pool, heads=2, dim=128, seed=8)
    share(b, [0, 12], [8990])
    check(b, 4, [0, 12], [8990], stride=True)
    b = Batch([1] * 2, [5000, 4321], page=16, pool=pool, heads=1, dim=64, seed=9)
    share(b, [0, 2], [4300])
    check(b, 8, [0, 2], [4300], scale=-0.2)
    b = Batch([333, 150], [3000, 2900], page=48, pool=pool, heads=1, dim=128, seed=10)
    share(b, [0, 2], [2640])
    check(b, 5, [0, 2], [2640], max_tokens=1)           # (the hint is not a limit)


@pytest.mark.parametrize("pool", ["bf16", "e4m3"])
@pytest.mark.parametrize("new", [1, 3, 30])
def test_long_own_contexts_are_divided(new, pool):
    """Few rows for the whole device: an item's own positions lie in many shares, each shorter than an item's cost."""
    for total, heads in (([6000, 5000], 1), ([1700, 2500], 2), ([2048 + 17, 900], 3)):
        b = Batch([new] * 2, total, page=16, pool=pool, heads=heads, dim=64, seed=17)
        share(b, [0, 2], [300])
        first = check(b, 4, [0, 2], [300])
        b = Batch([new] * 2, total, page=16, pool=pool, heads=heads, dim=64, seed=17)
        share(b, [0, 2], [300])
        again = check(b, 4, [0, 2], [300])
        assert all(torch.equal(x, y) for x, y in zip(first, again))


@pytest.mark.parametrize("rows,lens", [([0, 5], [300]), ([-1, 2], [300]), ([3, 1], [300]), ([0, 2, 1, 4], [300, 300, 300]),
                                       ([0, 4], [-3]), ([0, 4], [127]), ([2, 2], [300]), ([0], [])])
def test_groups_that_share_nothing(rows, lens):
    """The definition, within the same bounds: how a call divides its positions is its own (each division rounds the weights
    against other maxima), so bits may differ from spec_attend's."""
    b = Batch([2] * 4, [400, 380, 500, 420], page=16, heads=2, dim=64, seed=11)
    out, lse = check(b, 4, rows, lens)
    again, l2 = check(Batch([2] * 4, [400, 380, 500, 420], page=16, heads=2, dim=64, seed=11), 4, rows, lens)
    assert torch.equal(out, again) and torch.equal(lse, l2)


@pytest.mark.parametrize("pool", ["bf16", "e4m3"])
@pytest.mark.parametrize("new", [1, 40])
def test_bad_pages(pool, new):
    """A page that the first row's table lacks is left out for the whole group and flagged there; entries of other rows for
    shared positions are not read; an own page that is missing flags its row."""
    b = Batch([new, 0, new, new], [600, 600, 640, 700], page=16, pool=pool, heads=2, dim=64, seed=12, garbage=float("nan"))
    share(b, [0, 3], [512])
    b.table[0, 3] = b.pages
    b.table[2, 5] = -7                 # not read
    b.table[3, 40] = -1                # a row of no group
    check(b, 4, [0, 3], [512])
    b.table[0, :32] = -1               # nothing common is there
    check(b, 4, [0, 3], [512])
    b.table[2] = -1                    # and nothing of its own
    check(b, 4, [0, 3], [512])
    b.table = np.ascontiguousarray(b.table[:, :20])      # a cache longer than its table: each row is flagged
    check(b, 4, [0, 3], [512])


@pytest.mark.parametrize("pool", ["bf16", "e4m3"])
@pytest.mark.parametrize("new", [2, 40])
def test_values_that_are_not_finite(pool, new):
    """In common they reach all rows of the group, in a row's own positions the tokens that see them."""
    b = Batch([new, new, new], [400, 410, 420], page=16, pool=pool, heads=2, dim=64, seed=13)
    share(b, [0, 2], [256])

    def put(row, pos):
        page, slot = b.table[row, pos // 16], pos % 16
        if pool == "e4m3":
            b.exps[1, page, 1, slot] = 255
            b.values[1][page, 1, slot] = np.nan
        else:
            b.v[page, 1, slot, 5] = float("inf")
            b.values[1][page, 1, slot, 5] = np.inf

    put(1, 410 - 1)
    check(b, 4, [0, 2], [256])
    put(0, 100)
    check(b, 4, [0, 2], [256])


def test_workspace_serves_smaller_calls_streams_and_graphs():
    from speculative_decoding_verify_07_gb300 import binding as sv
    ws = sv.new_attend_shared_workspace(200, 40, 2, 4, 64, "cuda")
    for new, total, rows, lens in [([1] * 40, [300] * 40, [0, 20, 40], [256, 256]), ([50, 60], [900, 800], [0, 2], [640]),
                                   ([3] * 4, [200] * 4, [0, 4], [190]), ([1] * 40, [300] * 40, [0, 40], [256])]:
        b = Batch(new, total, page=16, heads=2, dim=64, seed=14)
        share(b, rows, lens)
        check(b, 4, rows, lens, workspace=ws)
    b = Batch([2] * 16, [1000] * 16, page=16, heads=2, dim=64, seed=15)
    share(b, [0, 16], [960])
    q = torch.randn((b.N, 8, 64), device="cuda").to(torch.bfloat16)
    args = dev(np.array([0, 16], np.int32)), dev(np.array([960], np.int32)), *b.args()
    want, lse = sv.spec_attend_shared(q, *args, max_tokens=2)
    out, l2 = torch.empty_like(want), torch.empty_like(lse)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            sv.spec_attend_shared(q, *args, max_tokens=2, out=out, lse=l2, workspace=ws, stream=side)
    for _ in range(5):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(l2, lse)
    small = sv.new_attend_shared_workspace(8, 16, 2, 4, 64, "cuda")
    with pytest.raises(sv.SpecError):
        sv.spec_attend_shared(q, *args, max_tokens=2, workspace=small)


def test_shared_is_as_close_to_spec_attend_as_either_to_the_oracle():
    from speculative_decoding_verify_07_gb300 import binding as sv
    b = Batch([3] * 32, [2100 + r for r in range(32)], page=16, heads=4, dim=128, seed=16)
    share(b, [0, 16, 32], [2048, 2000])
    q = torch.randn((b.N, 16, 128), device="cuda").to(torch.bfloat16)
    want, lse = sv.spec_attend(q, *b.args(), max_tokens=3)
    # (row 16's group shares 15 tiles of 128 of its 2000 positions)
    got, l2 = sv.spec_attend_shared(q, dev(np.array([0, 16, 32], np.int32)), dev(np.array([2048, 2000], np.int32)), *b.args(), max_tokens=3)
    assert (got.float() - want.float()).norm() <= 3 * BF16 * want.float().norm() and (l2 - lse).abs().max() <= 2e-5


def test_calls_at_once_and_one_after_the_other():
    """Two streams with a workspace each, and layers that follow one another on one workspace, eagerly and in a graph, with what
    reads a result right behind the call: the same bits as one call by itself."""
    from speculative_decoding_verify_07_gb300 import binding as sv
    jobs = []
    for seed, (new, total, rows, lens) in enumerate([([3] * 32, [3000 + 5 * r for r in range(32)], [0, 32], [2944]),
                                                     ([1] * 6, [900 + 40 * r for r in range(6)], [0, 3, 6], [768, 640])]):
        b = Batch(new, total, page=16, heads=4, dim=128, seed=30 + seed)
        share(b, rows, lens)
        q = torch.randn((b.N, 16, 128), device="cuda").to(torch.bfloat16)
        args = (q, dev(np.array(rows, np.int32)), dev(np.array(lens, np.int32)), *b.args())
        want = [t.clone() for t in sv.spec_attend_shared(*args, max_tokens=max(new))]
        jobs.append((args, max(new), want, sv.new_attend_shared_workspace(b.N, len(new), 4, 4, 128, "cuda"), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(20):
        got = []
        for args, most, _, ws, stream in jobs:
            with torch.cuda.stream(stream):
                out, lse = sv.spec_attend_shared(*args, max_tokens=most, workspace=ws)
                got.append((out + 0, lse + 0))
        torch.cuda.synchronize()
        for (a, b), job in zip(got, jobs):
            assert torch.equal(a, job[2][0]) and torch.equal(b, job[2][1])
    most_tokens, most_rows = max(j[0][0].shape[0] for j in jobs), max(len(j[0][4]) for j in jobs)
    ws = sv.new_attend_shared_workspace(most_tokens, most_rows, 4, 4, 128, "cuda")
    outs = [[torch.empty_like(t) for t in j[2]] for j in jobs]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for (args, most, _, _, _), (out, lse) in zip(jobs + jobs, outs + outs):
            sv.spec_attend_shared(*args, max_tokens=most, workspace=ws, out=out, lse=lse)
        copies = [[t + 0 for t in o] for o in outs]
    for _ in range(5):
        for o in outs + copies:
            for t in o:
                t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(t, w) for o, j in zip(copies, jobs) for t, w in zip(o, j[2]))
