"""The forward's operators over larger ranges: batches of more rows than a CTA has threads, and recurrences held to
the roundings that they still remember."""
import numpy as np
import pytest
import torch

from oracle import forward as of
from tests.test_gpu_forward import BF16, F32, Batch, check_attend, host

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")


@pytest.mark.parametrize("pool", ["bf16", "e4m3"])
@pytest.mark.parametrize("rows,most", [(129, 1), (257, 3), (513, 1), (513, 4096), (1100, 3), (1100, 4096)])
def test_attend_batches_of_many_rows(rows, most, pool):
    """Some rows without new tokens, some long; `most` chooses the kernel."""
    rng = np.random.default_rng(rows)
    new = rng.integers(0, 4, rows)
    new[[0, rows // 2, rows - 1]] = 0, 3, 2
    total = new + rng.integers(0, 40, rows)
    total[rows // 3] += 700
    check_attend(Batch(new.tolist(), total.tolist(), heads=1, dim=64, pool=pool, seed=rows), 2, max_tokens=most)


def remembered(g, size, back):
    """The bound on a state's error from the roundings of the tokens that it remembers: with e the error and H the state
    of |x|, e_t = a_t e_{t-1} + 2^-24 ((8 + 2 |g_t|) a_t H_{t-1} + 3 H_t).  exp(g) is off by 4 units and by |g| times
    the rounding of its argument; a multiply-add rounds once, and once more where tiles are joined."""
    a, out, e = np.exp(g), np.zeros_like(g), np.zeros(g.shape[::2])
    T = g.shape[1]
    with np.errstate(invalid="ignore"):
        slack = np.where(np.isneginf(g), 0.0, (8 + 2 * np.abs(g)) * a)
    order = reversed(range(T)) if back else range(T)
    before = np.zeros_like(e)
    for t in order:
        # backwards a token's decay acts on what comes out of it
        d = (t + 1 if t + 1 < T else None) if back else t
        at, st = (0.0, 0.0) if d is None else (a[:, d], slack[:, d])
        e = at * e + F32 * (st * before + 3 * size[:, t])
        out[:, t], before = e, size[:, t]
    return out


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,T,D,low,high", [(1, 20000, 40, -9.0, -4.0), (2, 9000, 256, -4.0, 0.0), (3, 700, 71, -2.0, 1.5), (2, 12, 64, -4.0, 0.0)])
def test_recur_errors_are_those_of_the_tokens_remembered(B, T, D, low, high, dtype):
    from speculative_decoding_verify_07_gb300 import binding as sv
    rng = np.random.default_rng(T)
    g = torch.from_numpy(-np.exp(rng.uniform(low, high, D) + 0.3 * rng.standard_normal((B, T, D)))).to(dtype)
    g[:, 5::997] = -torch.inf
    x, dh = (torch.from_numpy(rng.standard_normal((B, T, D))).to(dtype) for _ in range(2))
    h, last = sv.spec_recur(g.cuda(), x.cuda())
    dg, dx, ds = sv.spec_recur_backward(g.cuda(), h, dh.cuda())
    g64, x64, dh64, zero, lens = g.double().numpy(), x.double().numpy(), dh.double().numpy(), np.zeros((B, D)), np.full(B, T)
    rh, rlast = of.recur(g64, x64, zero, lens)
    hsize, _ = of.recur(g64, np.abs(x64), zero, lens)
    off = remembered(g64, hsize, False)
    assert (np.abs(host(h) - rh) <= off).all() and (np.abs(host(last) - rlast) <= off[:, -1]).all()
    rdg, rdx, rds = of.recur_backward(g64, host(h), dh64, zero, lens, zero)
    _, dsize, _ = of.recur_backward(g64, host(h), np.abs(dh64), zero, lens, zero)
    off = remembered(g64, dsize, True)
    out = F32 if dtype == torch.float32 else BF16
    assert (np.abs(host(dx) - rdx) <= off + out * np.abs(rdx)).all()
    assert (np.abs(host(ds) - rds) <= np.exp(g64[:, 0]) * (off[:, 0] + 8 * F32 * dsize[:, 0]) + 1e-37).all()
    hb = np.concatenate([zero[:, None], np.abs(host(h))[:, :-1]], 1)
    with np.errstate(invalid="ignore"):
        slack = np.where(np.isneginf(g64), 0.0, (8 + 2 * np.abs(g64)) * np.exp(g64))
    assert (np.abs(host(dg) - rdg) <= hb * (np.exp(g64) * off + F32 * slack * dsize) + out * np.abs(rdg) + 1e-37).all()


def test_recur_slow_decays_lean_to_no_side():
    """1000 remembered tokens of one sign: a decay that leans to one side by 1e-9 shows as 1e-6 in the mean.  The series
    leans by 1e-10 there, and the roundings of 64 channels and 20 memories (2^-25 a token at random) leave 3e-8."""
    from speculative_decoding_verify_07_gb300 import binding as sv
    rng = np.random.default_rng(1)
    g = (-1e-3 * rng.uniform(0.8, 1.2, (1, 20000, 64))).astype(np.float32)
    x = rng.uniform(0.5, 1.5, g.shape).astype(np.float32)
    h, _ = sv.spec_recur(torch.from_numpy(g).cuda(), torch.from_numpy(x).cuda())
    ref, _ = of.recur(g.astype(np.float64), x.astype(np.float64), np.zeros((1, 64)), [20000])
    assert abs(((host(h) - ref) / ref).mean()) <= 1e-6
