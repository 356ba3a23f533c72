"""Refusals of the forward's entry points, which need no GPU: arguments are checked before CUDA is touched."""
import os
import re

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 4096   # a fake, aligned address: never dereferenced
OK, NULL, DIM, DTYPE, ALIGN, WORKSPACE = 0, -1, -2, -3, -4, -5
REACHED = (-6, -7)      # all checks passed: there is no GPU here


@pytest.fixture(scope="module")
def sv():
    from speculative_decoding_verify_07_gb300 import build
    if not os.path.exists(build.LIB):
        build.build()
    from speculative_decoding_verify_07_gb300 import binding
    return binding


def no_gpu():
    if torch.cuda.is_available():
        pytest.skip("the calls would run")


def view(sv, **kw):
    a = dict(k=P, v=P, ke=None, ve=None, table=P, cu=P, kv=P, pstride=0, estride=0, pool=1, B=2, max_pages=3, pages=5,
             heads=2, ps=16, dim=64)
    a.update(kw)
    return sv.CACHE_T.pack(*(a[n] or 0 for n in ("k", "v", "ke", "ve", "table", "cu", "kv")), a["pstride"], a["estride"],
                           a["pool"], a["B"], a["max_pages"], a["pages"], a["heads"], a["ps"], a["dim"])


CACHE = [
    (dict(B=-1), DIM), (dict(pages=-1), DIM), (dict(max_pages=-1), DIM), (dict(heads=0), DIM), (dict(heads=65536), DIM),
    (dict(ps=0), DIM), (dict(ps=4097), DIM), (dict(dim=96), DIM), (dict(dim=256), DIM), (dict(max_pages=2 ** 30), DIM),
    (dict(pool=0), DTYPE), (dict(pool=7), DTYPE), (dict(pstride=-1), DIM), (dict(pstride=2 * 16 * 64 - 8), DIM),
    (dict(pool=2, ke=P, ve=P, estride=31), DIM), (dict(pool=2), NULL), (dict(pool=2, ke=P), NULL), (dict(cu=None), NULL),
    (dict(kv=None), NULL), (dict(table=None), NULL), (dict(k=None), NULL), (dict(v=None), NULL), (dict(cu=P + 2), ALIGN),
    (dict(table=P + 1), ALIGN), (dict(k=P + 8), ALIGN), (dict(v=P + 2), ALIGN), (dict(pstride=2 * 16 * 64 + 4), ALIGN),
    (dict(B=0), OK),
]


def write(sv, n=4, k=P, v=P, dtype=1, stride=0, flags=None, **kw):
    return sv.LIB.spec_cache_write(k, v, dtype, stride, n, view(sv, **kw), flags, None)


def attend(sv, n=4, q=P, out=P, lse=P, group=4, most=3, stride=0, flags=None, ws=P, wsb=1 << 40, **kw):
    return sv.LIB.spec_attend(q, stride, n, group, 0.1, most, view(sv, **kw), out, lse, flags, ws, wsb, None)


@pytest.mark.parametrize("kw,code", CACHE)
def test_cache_checks(sv, kw, code):
    assert write(sv, **kw) == code
    assert sv.LIB.spec_cache_read(P, P, 4, view(sv, **kw), None, None) == code
    assert attend(sv, **kw) == code


def test_calls_check_their_own_arguments(sv):
    assert sv.LIB.spec_cache_write(P, P, 1, 0, 4, None, None, None) == NULL
    assert write(sv, n=-1) == DIM
    assert write(sv, n=0, k=None) == OK
    assert write(sv, k=None) == NULL and write(sv, v=None) == NULL
    assert write(sv, dtype=2) == DTYPE
    assert write(sv, stride=-8) == DIM and write(sv, stride=2 * 64 - 1) == DIM
    assert write(sv, stride=2 * 64 + 4) == ALIGN and write(sv, k=P + 8) == ALIGN and write(sv, flags=P + 2) == ALIGN
    assert attend(sv, n=-1) == DIM and attend(sv, group=0) == DIM and attend(sv, group=65) == DIM
    assert attend(sv, most=-1) == DIM and attend(sv, stride=64) == DIM
    assert attend(sv, n=0, q=None) == OK
    assert attend(sv, q=None) == NULL and attend(sv, out=None) == NULL and attend(sv, ws=None) == NULL
    assert attend(sv, q=P + 2) == ALIGN and attend(sv, out=P + 8) == ALIGN and attend(sv, lse=P + 2) == ALIGN
    assert attend(sv, ws=P + 16) == ALIGN and attend(sv, wsb=8) == WORKSPACE
    assert sv.LIB.spec_attend_workspace_size(0, 4, 64) == 0 and sv.LIB.spec_attend_workspace_size(2, 65, 64) == 0
    assert sv.LIB.spec_attend_workspace_size(2, 4, 80) == 0 and sv.LIB.spec_attend_workspace_size(2, 4, 64) > 0


def test_valid_calls_reach_the_device(sv):
    no_gpu()
    assert write(sv) in REACHED and write(sv, dtype=0) in REACHED
    assert write(sv, pool=2, ke=P, ve=P) in REACHED
    assert sv.LIB.spec_cache_read(P, P, 4, view(sv, pool=2, ke=P, ve=P), None, None) in REACHED
    assert attend(sv) in REACHED and attend(sv, lse=None, most=4000) in REACHED
    assert recur(sv) in REACHED and backward(sv) in REACHED


def recur(sv, **kw):
    a = dict(g=P, gr=0, gt=0, x=P, dtype=1, state=P, slot=P, slots=4, lens=None, B=3, T=8, D=64, h=P, hd=0, last=P,
             ls=None, lss=3, flags=None, ws=P, wsb=1 << 40)
    a.update(kw)
    return sv.LIB.spec_recur(a["g"], a["gr"], a["gt"], a["x"], 0, 0, a["dtype"], a["state"], a["slot"], a["slots"],
                             a["lens"], a["B"], a["T"], a["D"], a["h"], a["hd"], a["last"], a["ls"], a["lss"], a["flags"],
                             a["ws"], a["wsb"], None)


def backward(sv, **kw):
    a = dict(g=P, h=P, hd=0, dh=P, dl=None, dtype=1, state=P, slot=P, slots=4, lens=None, B=3, T=8, D=64, dg=P, dx=P,
             ds=P, flags=None, ws=P, wsb=1 << 40)
    a.update(kw)
    return sv.LIB.spec_recur_backward(a["g"], 0, 0, a["h"], a["hd"], a["dh"], a["dl"], a["dtype"], a["state"], a["slot"],
                                      a["slots"], a["lens"], a["B"], a["T"], a["D"], a["dg"], a["dx"], a["ds"],
                                      a["flags"], a["ws"], a["wsb"], None)


def test_recur_checks(sv):
    for call in (recur, backward):
        assert call(sv, B=-1) == DIM and call(sv, T=-1) == DIM and call(sv, D=0) == DIM and call(sv, B=65536) == DIM
        assert call(sv, slots=-1) == DIM and call(sv, slot=None, slots=2) == DIM
        assert call(sv, dtype=2) == DTYPE and call(sv, hd=2) == DTYPE
        assert call(sv, B=0) == OK
        assert call(sv, g=None) == NULL and call(sv, h=None) == NULL and call(sv, ws=None) == NULL
        assert call(sv, g=P + 1) == ALIGN and call(sv, dtype=0, g=P + 2) == ALIGN and call(sv, h=P + 2) == ALIGN
        assert call(sv, state=P + 2) == ALIGN and call(sv, slot=P + 2) == ALIGN and call(sv, lens=P + 1) == ALIGN
        assert call(sv, flags=P + 2) == ALIGN and call(sv, ws=P + 16) == ALIGN and call(sv, wsb=0) == WORKSPACE
    assert recur(sv, x=None) == NULL and recur(sv, x=P + 1) == ALIGN and recur(sv, last=P + 2) == ALIGN
    assert recur(sv, lss=-1) == DIM and recur(sv, lss=2) == DIM
    assert backward(sv, dh=None) == NULL and backward(sv, dg=None) == NULL and backward(sv, dx=None) == NULL
    assert backward(sv, dh=P + 1) == ALIGN and backward(sv, ds=P + 2) == ALIGN and backward(sv, dl=P + 2) == ALIGN
    assert sv.LIB.spec_recur_workspace_size(-1, 2, 3) == 0 and sv.LIB.spec_recur_workspace_size(1, 1, 0) == 0


def test_every_declared_function_is_exported(sv):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "spec_forward.h")).read(), flags=re.S)
    names = re.findall(r"\b(spec_\w+)\s*\(", text)
    assert sorted(set(names)) == sorted(["spec_cache_write", "spec_cache_read", "spec_attend_workspace_size", "spec_attend",
                                         "spec_recur_workspace_size", "spec_recur", "spec_recur_backward"])
    for n in names:
        assert hasattr(sv.LIB, n)


def test_binding_refuses_tensors(sv):
    kv = torch.zeros((5, 2, 16, 64), dtype=torch.bfloat16)
    cu, ln, table = (torch.zeros(s, dtype=torch.int32) for s in ((3,), (2,), (2, 3)))
    q = torch.zeros((4, 8, 64), dtype=torch.bfloat16)
    new = torch.zeros((4, 2, 64), dtype=torch.bfloat16)

    def refuses(error, call, *a, **kw):
        with pytest.raises(error):
            call(*a, **kw)

    def bad_cache(error, *a):
        refuses(error, sv.spec_cache_write, new, new, *a)
        refuses(error, sv.spec_cache_read, 4, *a)
        refuses(error, sv.spec_attend, q, *a, max_tokens=1)

    bad_cache(TypeError, cu, ln, table, kv.float(), kv.float())
    bad_cache(ValueError, cu, ln, table, kv, kv[:4])
    bad_cache(ValueError, cu[:2], ln, table, kv, kv)
    bad_cache(TypeError, cu, ln.long(), table, kv, kv)
    bad_cache(ValueError, cu, ln, table, kv, kv, torch.zeros((5, 2, 16), dtype=torch.uint8), None)
    f8 = kv.to(torch.float8_e4m3fn)
    bad_cache(ValueError, cu, ln, table, f8, f8)
    bad_cache(ValueError, cu, ln, table, f8, f8, torch.zeros((5, 2, 15), dtype=torch.uint8), torch.zeros((5, 2, 16), dtype=torch.uint8))
    bad_cache(ValueError, cu, ln, table, kv.transpose(1, 2), kv.transpose(1, 2))     # not dense in a page
    refuses(ValueError, sv.spec_cache_write, new[:, :1], new[:, :1], cu, ln, table, kv, kv)
    refuses(ValueError, sv.spec_cache_write, new, new[:3], cu, ln, table, kv, kv)
    refuses(TypeError, sv.spec_cache_write, new.half(), new.half(), cu, ln, table, kv, kv)
    refuses(ValueError, sv.spec_cache_write, new, new, cu, ln, table, kv, kv, flags=torch.zeros(3, dtype=torch.int32))
    refuses(TypeError, sv.spec_attend, q.float(), cu, ln, table, kv, kv, max_tokens=1)
    refuses(ValueError, sv.spec_attend, q[:, :5], cu, ln, table, kv, kv, max_tokens=1)
    refuses(ValueError, sv.spec_attend, q, cu, ln, table, kv, kv, max_tokens=1, out=q[:2])
    refuses(ValueError, sv.new_attend_workspace, 2, 4, 80, "cpu")
    g = torch.zeros((2, 3, 8))
    refuses(ValueError, sv.spec_recur, g[0], g[0])
    refuses(TypeError, sv.spec_recur, g.half(), g.half())
    refuses(ValueError, sv.spec_recur, g, g.bfloat16())
    refuses(ValueError, sv.spec_recur, g.transpose(1, 2), g.transpose(1, 2))
    refuses(ValueError, sv.spec_recur, g, g, torch.zeros((2, 7)))
    refuses(TypeError, sv.spec_recur, g, g, torch.zeros((2, 8), dtype=torch.float64))
    refuses(ValueError, sv.spec_recur, g, g, None, torch.zeros(3, dtype=torch.int32))
    refuses(ValueError, sv.spec_recur_backward, g, g, g[:1])
    refuses(ValueError, sv.spec_recur_backward, g, g, g, d_last=torch.zeros((2, 7)))
