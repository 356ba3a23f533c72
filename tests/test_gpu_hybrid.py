"""GPU parity of the causal convolution and the selective scan with the float64 oracle.

Tolerances count roundings: half a step of bf16 is 2^-8 relative, of float32 2^-24.
"""
import numpy as np
import pytest
import torch

from oracle import forward as of
from oracle import hybrid as oh

pytestmark = pytest.mark.gpu

BF16, F32 = 2.0 ** -8, 2.0 ** -24
DT = [torch.bfloat16, torch.float32]


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")


def host(t):
    return t.detach().double().cpu().numpy()


def near(got, want, tol, what):
    bad = ~(np.abs(got - want) <= tol + 1e-37)
    assert not bad.any(), (what, np.argwhere(bad)[:5], got[bad][:5], want[bad][:5], np.broadcast_to(tol, got.shape)[bad][:5])


def half(dtype):
    return BF16 if dtype == torch.bfloat16 else F32


def padded(t, lens, wide=False):
    """The tensor on the device with NaN beyond each row's length; `wide`: as a slice of a larger projection."""
    t = t.clone()
    for r, n in enumerate(lens):
        t[r, n:] = float("nan")
    t = t.cuda()
    if wide:
        big = torch.full((t.shape[0], t.shape[1] + 1, *t.shape[2:-1], 2 * t.shape[-1] + 3), float("nan"), dtype=t.dtype, device="cuda")
        view = big[:, :t.shape[1], ..., 3:3 + t.shape[-1]]
        view.copy_(t)
        return view
    return t


# ---------------------------------------------------------------- convolution

def run_conv(B, T, C, width, dtype, silu=True, lens=None, state=True, bias=True, wide=False, states=False, seed=0):
    from speculative_decoding_verify_07_gb300 import binding as sv
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn((B, T, C), generator=gen).to(dtype)
    w, b = torch.randn((width, C), generator=gen), torch.randn((C,), generator=gen) if bias else None
    slots = B + 2
    st = torch.randn((slots, width - 1, C), generator=gen).to(dtype) if state else None
    slot = torch.randperm(slots, generator=gen)[:B].to(torch.int32) if state else None
    n = [T] * B if lens is None else lens
    ld = None if lens is None else torch.tensor(n, dtype=torch.int32, device="cuda")
    flags = torch.zeros(B, dtype=torch.int32, device="cuda")
    all_states = torch.full((B, T, width - 1, C), float("nan"), dtype=dtype, device="cuda") if states else None
    move = lambda t: None if t is None else t.cuda()
    y, last = sv.spec_conv(padded(x, n, wide), w.cuda(), move(b), move(st), move(slot), ld, silu=silu, states=all_states, flags=flags)
    torch.cuda.synchronize()
    assert not flags.any() and y.dtype == dtype and last.dtype == dtype
    first = np.zeros((B, width - 1, C)) if st is None else host(st)[slot.numpy()]
    wy, wl, ws, v, size = oh.conv(host(x), host(w), None if b is None else host(b), first, n, silu)
    # the sum's roundings (a tap each, and the bias) pass the gate with a slope below 1.1; the gate's own
    tol = half(dtype) * np.abs(wy) + 1.1 * (width + 1) * F32 * size + ((10 + 1.5 * np.abs(v)) * F32 * np.abs(wy) if silu else 0)
    near(host(y), wy, tol, "y")
    assert np.array_equal(host(last), wl)
    if states:
        assert np.array_equal(host(all_states), ws)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("width", [2, 3, 4, 5, 6, 7, 8])
@pytest.mark.parametrize("B,T,C", [(1, 1, 1), (3, 3, 64), (2, 33, 37), (2, 100, 1032)])
def test_conv(B, T, C, width, dtype):
    run_conv(B, T, C, width, dtype, seed=B + T + width, states=True)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("T", [2, 31, 32, 65])
def test_conv_lengths_strides_and_options(T, dtype):
    lens = [T, 0, 1, T // 2, T - 1]
    run_conv(5, T, 72, 4, dtype, lens=lens, states=True, seed=T)
    run_conv(5, T, 72, 4, dtype, lens=lens, wide=True, state=False, bias=False, silu=False, seed=T + 1)
    run_conv(5, T, 71, 8, dtype, lens=lens, wide=True, states=True, seed=T + 2)
    run_conv(5, T, 1024, 3, dtype, lens=lens, state=False, states=True, seed=T + 3)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("C", [40, 41])
def test_conv_in_place_in_pieces_is_the_whole(C, dtype):
    """A prompt in pieces, then single tokens, on a state updated in place, against one call: the same bits."""
    from speculative_decoding_verify_07_gb300 import binding as sv
    B, T, width = 3, 150, 4
    x, w = torch.randn((B, T, C), device="cuda").to(dtype), torch.randn((width, C), device="cuda")
    whole, last = sv.spec_conv(x, w)
    cache = torch.zeros((5, width - 1, C), dtype=dtype, device="cuda")
    slot = torch.tensor([4, 0, 2], dtype=torch.int32, device="cuda")
    cuts = [0, 1, 3, 70, 140, *range(141, T + 1)]
    got = [sv.spec_conv(x[:, a:e], w, None, cache, slot, last=cache, last_slot=slot)[0] for a, e in zip(cuts, cuts[1:])]
    assert torch.equal(torch.cat(got, 1), whole) and torch.equal(cache[slot.long()], last)
    assert not cache[[1, 3]].any()
    # no tokens at all: the state stays
    was = cache.clone()
    sv.spec_conv(x, w, None, cache, slot, torch.zeros(B, dtype=torch.int32, device="cuda"), last=cache, last_slot=slot)
    sv.spec_conv(x[:, :0], w, None, cache, slot, last=cache, last_slot=slot)
    assert torch.equal(cache, was)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("T", [3, 90])
def test_conv_bad_slots_are_flagged_and_left_alone(T, dtype):
    from speculative_decoding_verify_07_gb300 import binding as sv
    x, w = torch.ones((4, T, 16), device="cuda", dtype=dtype), torch.ones((4, 16), device="cuda")
    state = torch.ones((5, 3, 16), device="cuda", dtype=dtype)
    slot = torch.tensor([0, 5, -1, 2], dtype=torch.int32, device="cuda")
    to = torch.tensor([0, 1, 2, 9], dtype=torch.int32, device="cuda")
    flags, last = torch.zeros(4, dtype=torch.int32, device="cuda"), torch.full((6, 3, 16), 7.0, device="cuda", dtype=dtype)
    y, _ = sv.spec_conv(x, w, None, state, slot, silu=False, last=last, last_slot=to, flags=flags)
    assert flags.tolist() == [0] + [of.F_BAD_IDX] * 3
    assert (y[0] == 4).all() and not y[1:].any() and (last[0] == 1).all() and (last[1:] == 7).all()


def test_conv_what_is_not_finite_reaches_its_window_only():
    from speculative_decoding_verify_07_gb300 import binding as sv
    for bad in (float("nan"), float("inf")):
        x, w = torch.ones((1, 80, 24), device="cuda"), torch.ones((4, 24), device="cuda")
        x[0, 30, 5] = bad
        y, _ = sv.spec_conv(x, w, silu=False)
        there = torch.zeros((80, 24), dtype=torch.bool, device="cuda")
        there[30:34, 5] = True
        assert torch.equal(~torch.isfinite(y[0]), there)


# ----------------------------------------------------------------------- scan

def run_scan(B, T, D, N, dtype, groups=1, softplus=True, gate=True, skip=True, lens=None, state=True, wide=False, states=False,
             seed=0, slow=False, workspace=None):
    from speculative_decoding_verify_07_gb300 import binding as sv
    gen = torch.Generator().manual_seed(seed)
    normal = lambda *s: torch.randn(s, generator=gen)
    x, z = normal(B, T, D).to(dtype), normal(B, T, D).mul(3).to(dtype) if gate else None
    a = -torch.arange(1, N + 1) * torch.exp(0.1 * normal(D, N)) * (0.02 if slow else 1.0)
    step = torch.exp(torch.rand((D,), generator=gen) * np.log(100.0) + np.log(0.001))
    if softplus:
        dt, bias = (0.5 * normal(B, T, D)).to(dtype), step + torch.log(-torch.expm1(-step))
    else:
        dt, bias = (step * torch.exp(0.5 * normal(B, T, D))).to(dtype), None
    b, c = normal(B, T, groups, N).to(dtype), normal(B, T, groups, N).to(dtype)
    sk = normal(D) if skip else None
    slots = B + 2
    st = normal(slots, D, N) if state else None
    slot = torch.randperm(slots, generator=gen)[:B].to(torch.int32) if state else None
    n = [T] * B if lens is None else lens
    ld = None if lens is None else torch.tensor(n, dtype=torch.int32, device="cuda")
    flags = torch.zeros(B, dtype=torch.int32, device="cuda")
    all_states = torch.full((B, T, D, N), float("nan"), device="cuda") if states else None
    move = lambda t: None if t is None else t.cuda()
    put = lambda t: None if t is None else padded(t, n, wide)
    y, last = sv.spec_scan(put(x), put(dt), a.cuda(), put(b), put(c), move(sk), put(z), move(bias), move(st), move(slot), ld,
                           softplus=softplus, states=all_states, flags=flags, workspace=workspace)
    torch.cuda.synchronize()
    assert not flags.any() and y.dtype == dtype
    first = np.zeros((B, D, N)) if st is None else host(st)[slot.numpy()]
    opt = lambda t: None if t is None else host(t)
    wy, wl, ws, (ey, el, es) = oh.scan(host(x), host(dt), host(a), host(b), host(c), opt(sk), opt(z), opt(bias), first, n, softplus)
    near(host(last), wl, F32 * el, "last")
    near(host(y), wy, half(dtype) * np.abs(wy) + F32 * ey, "y")
    if states:
        near(host(all_states), ws, F32 * es, "states")
    for r in range(B):
        assert not y[r, n[r]:].any() and (not states or not all_states[r, n[r]:].any())


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("N", [8, 16, 32, 64, 128])
@pytest.mark.parametrize("B,T,D", [(1, 1, 1), (3, 3, 64), (2, 17, 33), (2, 100, 130), (1, 700, 40)])
def test_scan(B, T, D, N, dtype):
    run_scan(B, T, D, N, dtype, seed=B + T + N, states=T < 100)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("T", [3, 40, 300])
def test_scan_lengths_strides_and_options(T, dtype):
    lens = [T, 0, 1, T // 2, T - 1]
    run_scan(5, T, 72, 16, dtype, lens=lens, states=True, seed=T)
    run_scan(5, T, 72, 16, dtype, lens=lens, wide=True, state=False, gate=False, groups=2, seed=T + 1)
    run_scan(5, T, 69, 8, dtype, lens=lens, wide=True, softplus=False, skip=False, groups=3, seed=T + 2)
    run_scan(5, T, 70, 64, dtype, lens=lens, gate=False, skip=False, states=True, groups=70, seed=T + 3)


@pytest.mark.parametrize("dtype", DT)
def test_scan_long(dtype):
    """Splits of the tokens, slow decays: what the first tokens put in is there at the end."""
    run_scan(1, 6000, 48, 16, dtype, slow=True, seed=4)
    run_scan(2, 3000, 160, 8, dtype, slow=True, lens=[3000, 1025], groups=2, seed=5)
    run_scan(1, 2500, 24, 64, dtype, slow=True, state=False, seed=6)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("D", [64, 50])
@pytest.mark.parametrize("N", [8, 16, 64])
def test_scan_in_place_in_pieces_is_the_whole(N, D, dtype):
    """A prompt, then single steps on the cached state, against one call."""
    from speculative_decoding_verify_07_gb300 import binding as sv
    B, T = 3, 600
    gen = torch.Generator(device="cuda").manual_seed(N + D)
    normal = lambda *s: torch.randn(s, device="cuda", generator=gen)
    x, dt, z = (normal(B, T, D).to(dtype) for _ in range(3))
    b, c = normal(B, T, 1, N).to(dtype), normal(B, T, 1, N).to(dtype)
    a, skip = -0.05 - torch.rand((D, N), device="cuda", generator=gen), normal(D)
    whole, last = sv.spec_scan(x, dt, a, b, c, skip, z)
    cache, slot = torch.zeros((6, D, N), device="cuda"), torch.tensor([5, 0, 3], dtype=torch.int32, device="cuda")
    cuts = [0, 2, 400, 590, *range(591, T + 1)]
    got = []
    for s, e in zip(cuts, cuts[1:]):
        got.append(sv.spec_scan(x[:, s:e], dt[:, s:e], a, b[:, s:e], c[:, s:e], skip, z[:, s:e], None, cache, slot, last=cache,
                                last_slot=slot)[0])
    # the oracle's bound of either, on a state whose sum of magnitudes is below that of 40 tokens
    scale = float(last.abs().max())
    assert (cache[slot.long()] - last).abs().max() <= 200 * F32 * scale and not cache[[1, 2, 4]].any()
    got = torch.cat(got, 1)
    assert (got.double() - whole.double()).abs().max() <= (2 * half(dtype) + 1000 * F32) * float(whole.abs().max())
    was = cache.clone()
    sv.spec_scan(x, dt, a, b, c, skip, z, None, cache, slot, torch.zeros(B, dtype=torch.int32, device="cuda"), last=cache, last_slot=slot)
    sv.spec_scan(x[:, :0], dt[:, :0], a, b[:, :0], c[:, :0], skip, z[:, :0], None, cache, slot, last=cache, last_slot=slot)
    assert torch.equal(cache, was)


@pytest.mark.parametrize("T", [3, 700])
def test_scan_bad_slots_are_flagged_and_left_alone(T):
    from speculative_decoding_verify_07_gb300 import binding as sv
    B, D, N = 4, 32, 16
    one = torch.ones((B, T, D), device="cuda")
    b = torch.ones((B, T, 1, N), device="cuda")
    a, state = torch.full((D, N), -1.0, device="cuda"), torch.ones((5, D, N), device="cuda")
    slot = torch.tensor([0, 5, -1, 2], dtype=torch.int32, device="cuda")
    to = torch.tensor([0, 1, 2, 9], dtype=torch.int32, device="cuda")
    flags, last = torch.zeros(B, dtype=torch.int32, device="cuda"), torch.full((6, D, N), 7.0, device="cuda")
    y, _ = sv.spec_scan(one, one * 0, a, b, b, None, None, None, state, slot, softplus=False, last=last, last_slot=to, flags=flags)
    # delta 0: the state stays, y is its sum
    assert flags.tolist() == [0] + [of.F_BAD_IDX] * 3
    assert (y[0] == N).all() and not y[1:].any() and (last[0] == 1).all() and (last[1:] == 7).all()


@pytest.mark.parametrize("T", [5, 900])
def test_scan_graph_replays_are_the_same_bits(T):
    from speculative_decoding_verify_07_gb300 import binding as sv
    B, D, N = 2, 96, 16
    x, dt, z = (torch.randn((B, T, D), device="cuda").to(torch.bfloat16) for _ in range(3))
    b, c = (torch.randn((B, T, 1, N), device="cuda").to(torch.bfloat16) for _ in range(2))
    a = -torch.rand((D, N), device="cuda")
    w = torch.randn((4, D), device="cuda")
    ws = sv.new_scan_workspace(B, T, D, N, "cuda")
    u, conv_last = sv.spec_conv(x, w)
    want = [u, conv_last, *sv.spec_scan(u, dt, a, b, c, None, z, workspace=ws)]
    got = [torch.empty_like(t) for t in want]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sv.spec_conv(x, w, y=got[0], last=got[1])
        sv.spec_scan(got[0], dt, a, b, c, None, z, y=got[2], last=got[3], workspace=ws)
    for _ in range(4):
        for t in got:
            t.zero_()
        ws.fill_(255)       # (its contents need not be kept)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, want))


def test_scan_steps_of_any_size():
    """softplus from far below zero to far above; steps of zero and decays of zero."""
    from speculative_decoding_verify_07_gb300 import binding as sv
    v = torch.cat([torch.linspace(-80, 40, 4001), torch.linspace(-1, 1, 2001)])
    D, N = v.numel(), 8
    x = torch.ones((1, 1, D), device="cuda")
    a, b = torch.full((D, N), -1.0, device="cuda"), torch.ones((1, 1, 1, N), device="cuda")
    _, last = sv.spec_scan(x, v.cuda().view(1, 1, D), a, b, b)
    want = np.logaddexp(0.0, v.double().numpy())
    near(host(last)[0, :, 0], want, (12 + 1) * F32 * want, "softplus")       # its own bound and the product with 1
    # a huge step forgets the state and leaves what it puts in
    state = torch.full((1, 4, N), 3.0, device="cuda")
    one, big = torch.ones((1, 1, 4), device="cuda"), torch.full((1, 1, 4), 1e4, device="cuda")
    y, last = sv.spec_scan(one, big, a[:4], b, b, None, None, None, state, softplus=False)
    assert (last == 1e4).all() and (y == 1e4 * N).all()


def test_states_commit():
    """The convolution's and the scan's states a token are layers of spec_commit's verify buffers."""
    from speculative_decoding_verify_07_gb300 import binding as sv
    L, B, S, D, N, width, slots = 2, 5, 3, 64, 16, 4, 7
    gen = torch.Generator(device="cuda").manual_seed(3)
    normal = lambda *s: torch.randn(s, device="cuda", generator=gen)
    rec, conv = normal(L, slots, 1, D, N), normal(L, slots, width - 1, D).to(torch.bfloat16)
    slot = torch.tensor([6, 2, 0, 1, 4], dtype=torch.int32, device="cuda")
    u, dt, z = (normal(L, B, S, D).to(torch.bfloat16) for _ in range(3))
    b, c = (normal(L, B, S, 1, N).to(torch.bfloat16) for _ in range(2))
    w, a = normal(L, width, D), -torch.rand((L, D, N), device="cuda", generator=gen)
    vrec = torch.empty((L, B, S, 1, D, N), device="cuda")
    vconv = torch.empty((L, B, S, width - 1, D), dtype=torch.bfloat16, device="cuda")

    def layer(l, rows, count, **kw):
        x, cl = sv.spec_conv(u[l, rows, :count], w[l], None, conv0[l], slot[rows], states=kw.get("vconv"))
        _, rl = sv.spec_scan(x, dt[l, rows, :count], a[l], b[l, rows, :count], c[l, rows, :count], None, z[l, rows, :count], None,
                             rec0[l].view(slots, D, N), slot[rows], states=kw.get("vrec"))
        return cl, rl

    rec0, conv0 = rec.clone(), conv.clone()
    for l in range(L):
        layer(l, slice(None), S, vconv=vconv[l], vrec=vrec[l].view(B, S, D, N))
    accept = torch.tensor([1, 2, 3, 0, 2], dtype=torch.int32, device="cuda")
    sv.spec_commit(vrec, vconv, accept, slot, rec, conv)
    for l in range(L):
        for r in range(B):
            n = int(accept[r])
            cl, rl = layer(l, slice(r, r + 1), n) if n else (conv0[l, slot[r]][None], rec0[l, slot[r], 0][None])
            assert torch.equal(conv[l, slot[r]], cl[0]) and torch.equal(rec[l, slot[r], 0], rl[0])


def test_scans_at_once():
    """Split rows on two streams, a workspace each, and one workspace for calls one after the other: the same bits."""
    from speculative_decoding_verify_07_gb300 import binding as sv
    N, jobs = 16, []
    for B, T, D in ((1, 3000, 128), (2, 1500, 96)):
        x, dt, z = (torch.randn((B, T, D), device="cuda").to(torch.bfloat16) for _ in range(3))
        b, c = (torch.randn((B, T, 1, N), device="cuda").to(torch.bfloat16) for _ in range(2))
        args = (x, dt, -torch.rand((D, N), device="cuda"), b, c, None, z)
        jobs.append((args, [t.clone() for t in sv.spec_scan(*args)], sv.new_scan_workspace(B, T, D, N, "cuda"), torch.cuda.Stream()))
    largest = max((j[2] for j in jobs), key=lambda w: w.numel())
    torch.cuda.synchronize()
    for _ in range(20):
        got = []
        for args, _, ws, stream in jobs:
            with torch.cuda.stream(stream):
                got.append(sv.spec_scan(*args, workspace=ws))
        torch.cuda.synchronize()
        got += [sv.spec_scan(*args, workspace=largest) for args, _, _, _ in jobs]
        for g, job in zip(got, jobs + jobs):
            assert all(torch.equal(a, b) for a, b in zip(g, job[1]))
