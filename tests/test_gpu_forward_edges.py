"""The forward's operators where types, layouts and sizes end: scales of an 8-bit cache far apart, single-token
pages, streams, empty calls, and inputs whose alignment changes the path."""
import numpy as np
import pytest
import torch

from oracle import forward as of
from tests.test_gpu_forward import BF16, F32, Batch, check_attend, dev, host, run_recur

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")


def rescale(b, which, exps):
    """Gives a batch's keys (0) or values (1) these exponent bytes, and the oracle what they then stand for."""
    b.exps[which] = torch.from_numpy(exps.astype(np.uint8)).cuda()
    codes = (b.k, b.v)[which].view(torch.uint8).cpu().numpy()
    b.values[which] = of.cache_values(codes, exps)


def clear(b, which, pages, slots):
    """Zero vectors, as the cache writes them: zero codes under exponent byte 1."""
    (b.k, b.v)[which].view(torch.uint8)[pages, :, slots] = 0
    b.exps[which, pages, :, slots] = 1
    b.values[which][pages.cpu().numpy(), :, slots.cpu().numpy()] = 0.0


def places_of(b, row, positions):
    p = np.asarray(positions)
    return torch.from_numpy(b.table[row, p // b.page].astype(np.int64)).cuda(), torch.from_numpy(p % b.page).cuda()


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("new", [1, 3, 40])
def test_attend_zero_values_keep_their_weight(dim, new):
    """Positions whose value is zero count in the softmax however far their scale is from the others'."""
    total = 700
    b = Batch([new], [total], pool="e4m3", dim=dim, page=32, seed=31)
    one = [5, 333, total - new]
    rest = [p for p in range(total) if p not in one]
    for which in (0, 1):
        clear(b, which, *places_of(b, 0, rest))
    k = b.k.view(torch.uint8)
    pages, slots = places_of(b, 0, one)
    k[pages, :, slots] = 0x44                          # 3 in every dimension: scores of many sizes
    exps = b.exps[0].cpu().numpy()
    exps[pages.cpu().numpy(), :, slots.cpu().numpy()] = 127
    rescale(b, 0, exps)
    for group in (4, 1):
        check_attend(b, group)


@pytest.mark.parametrize("group", [4, 16])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("new", [2, 60])
@pytest.mark.parametrize("low,high", [(100, 135), (90, 150), (1, 130), (1, 221), (200, 221)])
def test_attend_values_of_all_scales(low, high, new, dim, group):
    b = Batch([new, 1], [400, 70], pool="e4m3", dim=dim, page=24, seed=low + high + new)
    rescale(b, 1, b.rng.integers(low, high + 1, b.exps[1].shape))
    rescale(b, 0, b.rng.integers(105, 122, b.exps[0].shape))
    check_attend(b, group)
    # the scales step by step along the row, up and down
    for order in (1, -1):
        exps = np.full(b.exps[1].shape, 127)
        for r, t in enumerate(b.kv_len):
            for p in range(t):
                exps[b.table[r, p // b.page], :, p % b.page] = np.linspace(low, high, t)[::order][p]
        rescale(b, 1, exps)
        check_attend(b, group)


@pytest.mark.parametrize("new", [3, 70])
@pytest.mark.parametrize("scale", [(0, 40), (180, 200)])
def test_attend_keys_of_all_scales(new, scale):
    b = Batch([new], [300], pool="e4m3", dim=128, page=16, seed=33)
    rescale(b, 0, b.rng.integers(*scale, b.exps[0].shape))
    # queries that bring the scores back to where weights differ
    check_attend(b, 4, q_size=2.0 ** (127 - 8 - scale[1]))


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("page", [1, 2, 3])
@pytest.mark.parametrize("new", [2, 90])
@pytest.mark.parametrize("pool", ["bf16", "e4m3"])
def test_attend_small_pages(pool, new, page, dim):
    check_attend(Batch([new, 1], [new + 77, 40], pool=pool, dim=dim, page=page, seed=34, garbage=float("nan"), interleave=True), 4)


@pytest.mark.parametrize("pool", ["bf16", "e4m3"])
@pytest.mark.parametrize("new", [3, 100])
def test_attend_zero_pool(pool, new):
    """A pool as it is allocated: zeros, and in 8 bits the exponent byte 0 too."""
    b = Batch([new], [200], pool=pool, dim=128, seed=35)
    b.k.zero_(), b.v.zero_()
    b.values[:] = 0
    if b.exps is not None:
        b.exps.zero_()
    out, lse = check_attend(b, 4)
    assert not out.any()


def test_empty_calls():
    from speculative_decoding_verify_07_gb300 import binding as sv
    b = Batch([0, 0], [40, 0], dim=64, seed=36)
    q = torch.empty((0, 4, 64), dtype=torch.bfloat16, device="cuda")
    out, lse = sv.spec_attend(q, *b.args(), max_tokens=0)
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)
    sv.spec_cache_write(q[:, :2], q[:, :2], *b.args())
    k, v = sv.spec_cache_read(0, *b.args())
    for B, T in ((0, 5), (2, 0)):
        state = torch.ones((3, 8), device="cuda")
        g = torch.zeros((B, T, 8), device="cuda")
        h, last = sv.spec_recur(g, g, state)
        dg, dx, ds = sv.spec_recur_backward(g, h, g, state, d_last=torch.ones((B, 8), device="cuda"))
        torch.cuda.synchronize()
        assert h.shape == (B, T, 8) and (last == 1).all() and (ds == 1).all()


@pytest.mark.parametrize("pool", ["bf16", "e4m3"])
def test_tokens_beyond_the_rows(pool):
    """Packed arrays longer than the rows' tokens: what is beyond them is not written."""
    from speculative_decoding_verify_07_gb300 import binding as sv
    b = Batch([3, 2], [50, 2], dim=64, pool=pool, seed=37)
    x = torch.randn((2, b.N + 6, b.heads, 64), device="cuda", dtype=torch.bfloat16)
    flags = torch.zeros(2, dtype=torch.int32, device="cuda")
    sv.spec_cache_write(x[0], x[1], *b.args(), flags=flags)
    q = torch.randn((b.N + 6, 4, 64), device="cuda", dtype=torch.bfloat16)
    want, wl = sv.spec_attend(q[: b.N].contiguous(), *b.args(), max_tokens=3)
    for most in (3, 300):
        out, lse = torch.full_like(q, 7), torch.full((b.N + 6, 4), 7.0, device="cuda")
        sv.spec_attend(q, *b.args(), max_tokens=most, out=out, lse=lse, flags=flags)
        assert (out[b.N:] == 7).all() and (lse[b.N:] == 7).all()
        assert (out[: b.N].float() - want.float()).abs().max() <= 4 * BF16 * want.float().abs().max()
    k, v = sv.spec_cache_read(b.N + 6, *b.args(), flags=flags)
    assert not k[b.N:].any() and not v[b.N:].any() and not flags.any()


def test_cache_and_recurrence_on_another_stream():
    from speculative_decoding_verify_07_gb300 import binding as sv
    side = torch.cuda.Stream()
    b = Batch([300, 3], [700, 70], dim=128, pool="e4m3", seed=38)
    args = b.args()
    x = torch.randn((2, b.N, b.heads, 128), device="cuda", dtype=torch.bfloat16)
    g = -torch.rand((2, 3000, 136), device="cuda").to(torch.bfloat16)
    y, dh = (torch.randn((2, 3000, 136), device="cuda").to(torch.bfloat16) for _ in range(2))
    sv.spec_cache_write(x[0], x[1], *args)
    want = list(sv.spec_cache_read(b.N, *args))
    h, last = sv.spec_recur(g, y)
    want += [h, last, *sv.spec_recur_backward(g, h, dh)]
    b.k.view(torch.uint8).zero_(), b.v.view(torch.uint8).zero_()
    side.wait_stream(torch.cuda.current_stream())
    sv.spec_cache_write(x[0], x[1], *args, stream=side)
    got = list(sv.spec_cache_read(b.N, *args, stream=side))
    h, last = sv.spec_recur(g, y, stream=side)
    got += [h, last, *sv.spec_recur_backward(g, h, dh, stream=side)]
    side.synchronize()
    assert all(torch.equal(a, c) for a, c in zip(got, want))


@pytest.mark.parametrize("T", [5, 700])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_recur_any_alignment_gives_the_same_bits(T, dtype):
    """Inputs that begin between 16-byte boundaries, broadcast rows and tokens: the values decide alone."""
    from speculative_decoding_verify_07_gb300 import binding as sv
    B, D = 3, 72
    g = -torch.rand((1, 1, D), device="cuda").to(dtype)
    x = torch.randn((B, T, D), device="cuda").to(dtype)
    full = g.expand(B, T, D).contiguous()
    h, last = sv.spec_recur(full, x, h_dtype=dtype)
    grads = sv.spec_recur_backward(full, h, x)
    odd = torch.zeros(B * T * D + 1, dtype=dtype, device="cuda")
    odd[1:] = x.flatten()
    for gg, xx in ((full, odd[1:].view(B, T, D)), (g.expand(B, T, D), x)):
        h2, last2 = sv.spec_recur(gg, xx, h_dtype=dtype)
        assert torch.equal(h2, h) and torch.equal(last2, last)
        for a, c in zip(sv.spec_recur_backward(gg, h2, xx), grads):
            assert torch.equal(a, c)


def test_recur_gradients_against_differences():
    """Directional derivatives of sum(h . dh) + sum(last . d_last) against central differences in float64."""
    from speculative_decoding_verify_07_gb300 import binding as sv
    rng = np.random.default_rng(40)
    B, T, D = 2, 600, 16
    g, x, dh = -rng.random((B, T, D)), rng.standard_normal((B, T, D)), rng.standard_normal((B, T, D))
    first, d_last = rng.standard_normal((B, D)), rng.standard_normal((B, D))
    g, x, dh, first, d_last = (a.astype(np.float32).astype(np.float64) for a in (g, x, dh, first, d_last))
    f = lambda a: torch.from_numpy(a.astype(np.float32)).cuda()
    h, _ = sv.spec_recur(f(g), f(x), f(first))
    dg, dx, ds = (host(t) for t in sv.spec_recur_backward(f(g), h, f(dh), f(first), d_last=f(d_last)))

    def loss(g, x, first):
        hh, last = of.recur(g, x, first, np.full(B, T))
        return (hh * dh).sum() + (last * d_last).sum()

    for grad, at in ((dg, 0), (dx, 1), (ds, 2)):
        for _ in range(3):
            way = rng.standard_normal(grad.shape)
            eps = 1e-4
            args = [g, x, first]
            up, down = list(args), list(args)
            up[at], down[at] = args[at] + eps * way, args[at] - eps * way
            want = (loss(*up) - loss(*down)) / (2 * eps)
            # float32 sums of about 1 / (1 - exp(g)) remembered tokens, and eps^2 of the difference's third derivative
            assert abs((grad * way).sum() - want) <= 64 * F32 * np.abs(grad * way).sum() + 1e-5 * np.abs(grad * way).sum()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T", [31, 32, 33, 128, 129, 2048, 2049])
def test_recur_lengths_around_the_tiles(T, dtype):
    run_recur(2, T, 64, dtype, dtype, seed=T, lens=[T, T - 1])


@pytest.mark.parametrize("N", [1, 2, 300, 1200, 1217, 4865])
@pytest.mark.parametrize("heads", [1, 3, 8, 33])
def test_cache_any_number_of_heads_and_tokens(N, heads):
    from speculative_decoding_verify_07_gb300 import binding as sv
    rng = np.random.default_rng(N + heads)
    cuts = np.sort(rng.integers(0, N + 1, 3))
    new = np.diff(np.concatenate([[0], cuts, [N]])).tolist()
    b = Batch(new, [n + 5 for n in new], heads=heads, dim=64, page=16, pool="e4m3", seed=N)
    x = torch.from_numpy(rng.standard_normal((2, N, heads, 64))).to(torch.bfloat16)
    sv.spec_cache_write(x[0].cuda(), x[1].cuda(), *b.args())
    got = sv.spec_cache_read(N, *b.args())
    for a, c in zip(x, got):
        codes, exps, _ = of.quantise(a.double().numpy())
        assert np.array_equal(host(c), of.cache_values(codes, exps))
