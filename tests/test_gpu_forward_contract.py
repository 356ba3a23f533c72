"""What spec_forward.h promises beside the values: states updated in place, flags, answers that no hint and no
neighbour changes."""
import numpy as np
import pytest
import torch

from oracle import forward as of
from tests.test_gpu_forward import Batch, check_attend

pytestmark = pytest.mark.gpu

DT = [torch.bfloat16, torch.float32]


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")


def scan_inputs(B, T, D, dtype, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    # what a row begins with is still seen at its end: decays of 1 / T a token
    g = (-torch.rand((B, T, D), device="cuda", generator=gen) / T).to(dtype)
    x, dh = (torch.randn((B, T, D), device="cuda", generator=gen).to(dtype) for _ in range(2))
    return g, x, dh, 100 * torch.randn((B + 3, D), device="cuda", generator=gen)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("tiles", [2, 16, 17, 40])
@pytest.mark.parametrize("B,D", [(3, 71), (4, 136), (6, 1024)])
def test_recur_in_place_is_the_call_out_of_place(B, D, tiles, dtype):
    """`last` over `state`: every tile of a long row sees the state that was there before the call."""
    from speculative_decoding_verify_07_gb300 import binding as sv
    T = tiles * (128 if dtype == torch.bfloat16 else 64) - 3
    g, x, _, state = scan_inputs(B, T, D, dtype, tiles + B)
    slot = torch.randperm(B + 3, device="cuda")[:B].to(torch.int32)
    ws = sv.new_recur_workspace(B, T, D, "cuda")
    h, last = sv.spec_recur(g, x, state, slot, h_dtype=dtype, workspace=ws)
    want = state.clone()
    want[slot.long()] = last
    got = torch.empty_like(h)
    for _ in range(25):
        cache = state.clone()
        sv.spec_recur(g, x, cache, slot, h=got, last=cache, last_slot=slot, workspace=ws)
        assert torch.equal(got, h) and torch.equal(cache, want)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("tiles", [1, 2, 17, 40])
def test_recur_backward_in_place_is_the_call_out_of_place(tiles, dtype):
    """`d_state` over `d_last`."""
    from speculative_decoding_verify_07_gb300 import binding as sv
    B, D, T = 5, 520, tiles * (128 if dtype == torch.bfloat16 else 64) - 3
    g, x, dh, state = scan_inputs(B, T, D, dtype, tiles)
    h, _ = sv.spec_recur(g, x, state[:B])
    want = sv.spec_recur_backward(g, h, dh, state[:B], d_last=state[3:])
    for _ in range(25):
        both = state[3:].clone()
        got = sv.spec_recur_backward(g, h, dh, state[:B], d_last=both, d_state=both)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("pool", ["bf16", "e4m3"])
@pytest.mark.parametrize("new", [2, 150])          # either kernel
@pytest.mark.parametrize("wide", [9, 4, 1, 0])     # pages of the table: row 0 ends in page 10, row 1 in page 3
def test_attend_flags_a_cache_longer_than_its_page_table(wide, new, pool):
    b = Batch([new, 1, 0], [11 * 16 - 3, 3 * 16 + 5, 160], page=16, pool=pool, seed=41)
    b.table = np.ascontiguousarray(b.table[:, :wide])
    check_attend(b, 4, expect_flags=np.array([of.F_BAD_IDX, of.F_BAD_IDX if wide < 4 else 0, 0], np.uint32))


@pytest.mark.parametrize("byte", [221, 222, 246, 254, 255])
@pytest.mark.parametrize("new,most", [(3, 3), (3, 4096), (140, 140), (140, 1)])     # either kernel, either hint
@pytest.mark.parametrize("dim", [64, 128])
def test_attend_takes_the_largest_scales_for_nan_in_either_kernel(dim, new, most, byte):
    b = Batch([new, 1], [new + 70, 40], page=16, pool="e4m3", dim=dim, seed=42)
    at = 70 + new // 2
    page, slot = b.table[0, at // 16], at % 16
    b.exps[1, page, :, slot] = byte
    codes = b.v.view(torch.uint8)[page, :, slot].cpu().numpy()
    b.values[1][page, :, slot] = of.cache_values(codes, np.full(b.heads, byte)) if byte <= 221 else np.nan
    out, _ = check_attend(b, 4, max_tokens=most)
    assert out[new // 2:new].isnan().all() == (byte > 221) and torch.isfinite(out[:new // 2]).all()


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("tiles", [38, 42, 50])      # 608, 672 and 800 in all: as many CTAs as run at once, and more
def test_recur_alignment_changes_no_bits_of_long_rows(tiles, dtype):
    from speculative_decoding_verify_07_gb300 import binding as sv
    B, D, T = 1, 1024, tiles * (128 if dtype == torch.bfloat16 else 64)
    g, x, dh, state = scan_inputs(B, T, D, dtype, tiles)

    def shifted(t):          # begins between 16-byte boundaries
        odd = torch.zeros(t.numel() + 1, dtype=t.dtype, device="cuda")
        odd[1:] = t.flatten()
        return odd[1:].view(t.shape)

    h, last = sv.spec_recur(g, x, state[:1])
    h2, last2 = sv.spec_recur(shifted(g), shifted(x), state[:1])
    assert torch.equal(h2, h) and torch.equal(last2, last)
    for a, b in zip(sv.spec_recur_backward(shifted(g), h, dh, state[:1]), sv.spec_recur_backward(g, h, dh, state[:1])):
        assert torch.equal(a, b)


@pytest.mark.parametrize("kv_len", [0, -1, -2 ** 31, -2 ** 31 + 2])
@pytest.mark.parametrize("new", [3, 150])
def test_rows_of_negative_length_hold_nothing(new, kv_len):
    from speculative_decoding_verify_07_gb300 import binding as sv
    b = Batch([new, 2], [new + 40, 30], page=16, seed=43)
    b.kv_len[0] = kv_len
    check_attend(b, 4, expect_flags=np.zeros(2, np.uint32))
    before = b.k.clone()
    flags = torch.zeros(2, dtype=torch.int32, device="cuda")
    x = torch.ones((b.N, b.heads, b.dim), dtype=torch.bfloat16, device="cuda")
    sv.spec_cache_write(x, x, *b.args(), flags=flags)
    assert flags.tolist() == [of.F_BAD_IDX, 0]
    assert (b.k != before).flatten(1).any(1).sum() == 1          # row 1's two tokens, positions 28 and 29


# tiles of 16 and 32 query rows in the few-rows kernel, and of 128
@pytest.mark.parametrize("new,group,pool", [(3, 4, "bf16"), (1, 2, "bf16"), (9, 5, "bf16"), (40, 4, "bf16"), (40, 4, "e4m3"),
                                            (3, 4, "e4m3"), (1, 2, "e4m3"), (9, 5, "e4m3")])
@pytest.mark.parametrize("high,low", [(100, -100), (60, 0), (40, -20)])
def test_attend_a_query_is_not_measured_by_its_neighbours(high, low, new, group, pool):
    """Queries of one row and head group that are far apart in size, as an unused token's may be: each keeps its bits."""
    b = Batch([new, 2], [new + 200, 130], page=16, pool=pool, dim=128, seed=44)
    size = np.full((b.N, b.heads * group, 1), 2.0)
    size[::2, ::group] = 2.0 ** high
    size[::3, group - 1::group] = 2.0 ** low
    check_attend(b, group, q_size=size)


@pytest.mark.parametrize("new,most", [(3, 3), (150, 150)])
def test_exponent_byte_zero_is_read_as_one(new, most):
    """By the read and by both attention kernels, for keys and values: the header's one case apart from c 2^(e - 127)."""
    from speculative_decoding_verify_07_gb300 import binding as sv
    b = Batch([new], [new + 60], page=16, pool="e4m3", dim=64, seed=46)
    q = (2.0 ** 120 * torch.randn((b.N, 8, 64), device="cuda")).to(torch.bfloat16)
    got = []
    for byte in (0, 1):
        b.exps.fill_(byte)
        got.append([*sv.spec_cache_read(b.N, *b.args()), *sv.spec_attend(q, *b.args(), max_tokens=most)])
    assert all(torch.equal(a, c) for a, c in zip(*got)) and got[0][0].any() and got[0][2].any()
    codes = b.k.view(torch.uint8).cpu().numpy()
    _, _, _, page, slot = b.places()[0]
    assert np.array_equal(got[0][0][0].double().cpu().numpy(), of.e4m3_value(codes[page, :, slot]) * 2.0 ** -126)


@pytest.fixture(scope="module")
def late(tmp_path_factory):
    """The library with waits whose bound is zero, so that every wait which waits at all passes it."""
    from speculative_decoding_verify_07_gb300 import binding, build
    at = tmp_path_factory.mktemp("late")
    return binding._load(build.build(defines=("SPEC_WAIT_NS=0",), lib=str(at / "lib" / "liblate.so"), objdir=str(at / "obj")))


def flagged_late(flags):
    assert not (flags & ~256).any()
    return bool((flags & 256).any())


@pytest.mark.parametrize("pool", ["bf16", "e4m3"])
@pytest.mark.parametrize("rows,new,total", [(40, 3, 8000), (2, 300, 3000), (1, 30, 60000)])
@pytest.mark.parametrize("dim", [64, 128])
def test_attend_a_late_wait_is_flagged_and_ends_in_order(late, monkeypatch, dim, rows, new, total, pool):
    """What passes its bound is reported; its copies are still waited for, and the workspace serves on."""
    from speculative_decoding_verify_07_gb300 import binding as sv
    page, heads = 64, 4
    pages = rows * -(-total // page)
    pools = torch.randn((2, pages, heads, page, dim), device="cuda").to(torch.bfloat16)
    exps = (None, None)
    if pool == "e4m3":
        pools = pools.float().to(torch.float8_e4m3fn)
        exps = torch.full((2, pages, heads, page), 127, dtype=torch.uint8, device="cuda")
    table = torch.randperm(pages, device="cuda").to(torch.int32).view(rows, -1)
    args = (new * torch.arange(rows + 1, device="cuda", dtype=torch.int32), torch.full((rows,), total, dtype=torch.int32, device="cuda"),
            table, *pools, *exps)
    q = torch.randn((rows * new, 4 * heads, dim), device="cuda", dtype=torch.bfloat16)
    ws = sv.new_attend_workspace(heads, 4, dim, "cuda")
    call = dict(max_tokens=new, workspace=ws)
    want = sv.spec_attend(q, *args, **call)
    flags = torch.zeros(rows, dtype=torch.int32, device="cuda")
    with monkeypatch.context() as m:
        m.setattr(sv, "LIB", late)
        got = sv.spec_attend(q, *args, **call, flags=flags)
    # (few rows of short vectors, or of 8 bits, take longer to compute than to copy)
    assert flagged_late(flags) or (4 * new <= 64 and (dim == 64 or pool == "e4m3"))
    assert all(torch.equal(a, c) for a, c in zip(got, want))
    flags.zero_()
    again = sv.spec_attend(q, *args, **call, flags=flags)
    assert not flags.any() and all(torch.equal(a, c) for a, c in zip(again, want))


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("T", [100, 3000])
def test_recur_a_late_wait_is_flagged_and_ends_in_order(late, monkeypatch, T, dtype):
    from speculative_decoding_verify_07_gb300 import binding as sv
    B, D = 3, 512
    g, x, dh, state = scan_inputs(B, T, D, dtype, T)
    ws, flags = sv.new_recur_workspace(B, T, D, "cuda"), torch.zeros((2, B), dtype=torch.int32, device="cuda")

    def both(f=(None, None)):
        h, last = sv.spec_recur(g, x, state[:B], workspace=ws, flags=f[0])
        return [h, last, *sv.spec_recur_backward(g, h, dh, state[:B], workspace=ws, flags=f[1])]

    want = both()
    with monkeypatch.context() as m:
        m.setattr(sv, "LIB", late)
        got = both(flags)
    assert flagged_late(flags[0]) and flagged_late(flags[1])
    assert all(torch.equal(a, c) for a, c in zip(got, want))
    flags.zero_()
    assert all(torch.equal(a, c) for a, c in zip(both(flags), want)) and not flags.any()
