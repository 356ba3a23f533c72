"""Refusals of the hybrid mixers, which need no GPU: arguments are checked before CUDA is touched."""
import os
import re

import pytest
import torch

from tests.test_forward_abi_cpu import CACHE, view

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


def conv(sv, **kw):
    a = dict(x=P, weight=P, bias=P, state=P, slot=P, lens=P, y=P, states=P, last=P, last_slot=P, flags=P, x_row=24, x_tok=8,
             dtype=1, B=3, T=3, C=8, width=4, slots=4, last_slots=4, silu=1)
    assert not set(kw) - set(a)
    a.update(kw)
    return sv.LIB.spec_conv(sv.CONV_T.pack(*(v or 0 for v in a.values())), None)


def scan(sv, ws=P, wsb=1 << 40, **kw):
    a = dict(x=P, dt=P, z=P, b=P, c=P, a=P, skip=P, dt_bias=P, state=P, slot=P, lens=P, y=P, states=P, last=P, last_slot=P, flags=P)
    a.update({n: 16 for n in ("x_row", "x_tok", "dt_row", "dt_tok", "z_row", "z_tok", "b_row", "b_tok", "b_group", "c_row", "c_tok",
                              "c_group")})
    a.update(dtype=1, B=3, T=3, D=8, N=16, groups=2, slots=4, last_slots=4, softplus=1)
    assert not set(kw) - set(a)
    a.update(kw)
    return sv.LIB.spec_scan(sv.SCAN_T.pack(*(v or 0 for v in a.values())), ws, wsb, None)


BOTH = [(dict(B=-1), DIM), (dict(B=65536), DIM), (dict(T=-1), DIM), (dict(slots=-1), DIM), (dict(last_slots=-1), DIM),
        (dict(slot=None, slots=2), DIM), (dict(last_slot=None, last_slots=2), DIM), (dict(dtype=2), DTYPE), (dict(dtype=-1), DTYPE),
        (dict(T=0x7fffff01), DIM), (dict(slot=P + 2), ALIGN), (dict(last_slot=P + 1), ALIGN), (dict(lens=P + 2), ALIGN),
        (dict(flags=P + 2), ALIGN), (dict(x=None), NULL), (dict(y=None), NULL), (dict(x=P + 1), ALIGN), (dict(y=P + 1), ALIGN),
        (dict(dtype=0, x=P + 2), ALIGN), (dict(state=P + 1), ALIGN), (dict(states=P + 1), ALIGN), (dict(last=P + 1), ALIGN),
        (dict(B=0, x=None), OK), (dict(T=0, last=None, x=None), OK)]


@pytest.mark.parametrize("kw,code", BOTH)
def test_checks_of_both(sv, kw, code):
    assert conv(sv, **kw) == code and scan(sv, **kw) == code


def test_conv_checks(sv):
    assert sv.LIB.spec_conv(None, None) == NULL
    assert conv(sv, C=0) == DIM and conv(sv, C=(1 << 26) + 1) == DIM and conv(sv, width=1) == DIM and conv(sv, width=9) == DIM
    assert conv(sv, weight=None) == NULL and conv(sv, weight=P + 2) == ALIGN and conv(sv, bias=P + 2) == ALIGN


def test_scan_checks(sv):
    assert sv.LIB.spec_scan(None, P, 1 << 40, None) == NULL
    assert scan(sv, D=0) == DIM and scan(sv, D=(1 << 24) + 2) == DIM and scan(sv, groups=0) == DIM and scan(sv, groups=3) == DIM
    for n in (0, 4, 15, 24, 256):
        assert scan(sv, N=n) == DIM and sv.LIB.spec_scan_workspace_size(1, 1, 8, n) == 0
    for name in ("dt", "b", "c", "a"):
        assert scan(sv, **{name: None}) == NULL
    for name in ("dt", "z", "b", "c"):
        assert scan(sv, **{name: P + 1}) == ALIGN
    for name in ("a", "state", "states", "last"):
        assert scan(sv, **{name: P + 8}) == ALIGN
    assert scan(sv, skip=P + 2) == ALIGN and scan(sv, dt_bias=P + 2) == ALIGN
    assert scan(sv, ws=None) == NULL and scan(sv, ws=P + 16) == ALIGN and scan(sv, wsb=8) == WORKSPACE
    assert sv.LIB.spec_scan_workspace_size(-1, 1, 8, 16) == 0 and sv.LIB.spec_scan_workspace_size(1, 1, 0, 16) == 0
    assert sv.LIB.spec_scan_workspace_size(1, 1, 8, 16) >= 256


def shared(sv, n=4, q=P, rows=P, lens=P, groups=2, out=P, lse=P, group=4, most=3, stride=0, flags=None, ws=P, wsb=1 << 40, **kw):
    return sv.LIB.spec_attend_shared(q, stride, n, group, 0.1, most, view(sv, **kw), rows, lens, groups, out, lse, flags, ws, wsb, None)


@pytest.mark.parametrize("kw,code", CACHE)
def test_shared_checks_the_cache(sv, kw, code):
    assert shared(sv, **{"groups": 0, **kw} if kw.get("B") == 0 else kw) == code


def test_shared_checks(sv):
    assert shared(sv, n=-1) == DIM and shared(sv, group=0) == DIM and shared(sv, group=65) == DIM and shared(sv, most=-1) == DIM
    assert shared(sv, stride=64) == DIM and shared(sv, groups=-1) == DIM and shared(sv, groups=3) == DIM
    assert shared(sv, n=0, q=None) == OK
    for name in ("q", "rows", "lens", "out", "ws"):
        assert shared(sv, **{name: None}) == NULL
    assert shared(sv, q=P + 2) == ALIGN and shared(sv, out=P + 8) == ALIGN and shared(sv, lse=P + 2) == ALIGN
    assert shared(sv, rows=P + 2) == ALIGN and shared(sv, lens=P + 1) == ALIGN and shared(sv, flags=P + 2) == ALIGN
    assert shared(sv, ws=P + 16) == ALIGN
    size = sv.LIB.spec_attend_shared_workspace_size
    assert shared(sv, wsb=size(4, 2, 2, 4, 64) - 1) == WORKSPACE
    assert size(-1, 2, 2, 4, 64) == 0 and size(4, -1, 2, 4, 64) == 0 and size(4, 2, 0, 4, 64) == 0 and size(4, 2, 2, 65, 64) == 0
    assert size(4, 2, 2, 4, 80) == 0 and size(4, 2, 65535, 2, 64) == 0
    assert size(4, 2, 2, 4, 64) >= sv.LIB.spec_attend_workspace_size(2, 4, 64) + 4 * 8 * 65 * 4


def test_valid_calls_reach_the_device(sv):
    if torch.cuda.is_available():
        pytest.skip("the calls would run")
    none = {n: None for n in ("state", "slot", "lens", "states", "last_slot", "flags")}
    assert conv(sv) in REACHED and conv(sv, **none, bias=None, dtype=0, silu=0) in REACHED and conv(sv, T=0, x=None) in REACHED
    assert shared(sv) in REACHED and shared(sv, rows=None, lens=None, groups=0) in REACHED
    assert scan(sv) in REACHED and scan(sv, **none, z=None, skip=None, dt_bias=None, dtype=0) in REACHED


def test_every_declared_function_is_exported(sv):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "spec_hybrid.h")).read(), flags=re.S)
    names = set(re.findall(r"\b(spec_\w+)\s*\(", text))
    assert {"spec_conv", "spec_scan", "spec_scan_workspace_size", "spec_attend_shared", "spec_attend_shared_workspace_size"} == names
    for n in names:
        assert hasattr(sv.LIB, n)


def test_binding_refuses_tensors(sv):
    x, w = torch.zeros((2, 3, 8)), torch.zeros((4, 8))

    def refuses(error, call, *a, **kw):
        with pytest.raises(error):
            call(*a, **kw)

    refuses(ValueError, sv.spec_conv, x[0], w)
    refuses(ValueError, sv.spec_conv, x, w[0])
    refuses(ValueError, sv.spec_conv, x, w[:1])
    refuses(ValueError, sv.spec_conv, x, torch.zeros((9, 8)))
    refuses(TypeError, sv.spec_conv, x.half(), w)
    refuses(TypeError, sv.spec_conv, x, w.bfloat16())
    refuses(ValueError, sv.spec_conv, x, w[:, :7])
    refuses(ValueError, sv.spec_conv, x.transpose(1, 2), torch.zeros((4, 3)))
    refuses(ValueError, sv.spec_conv, x, w, torch.zeros(7))
    refuses(TypeError, sv.spec_conv, x, w, None, None, torch.zeros(2))
    refuses(ValueError, sv.spec_conv, x, w)                                      # on the host
    s = dict(x=x, dt=x, a=torch.zeros((8, 16)), b=torch.zeros((2, 3, 1, 16)), c=torch.zeros((2, 3, 1, 16)))
    refuses(ValueError, sv.spec_scan, **{**s, "x": x[0]})
    refuses(ValueError, sv.spec_scan, **{**s, "dt": x.bfloat16()})
    refuses(ValueError, sv.spec_scan, **{**s, "dt": x[:, :2]})
    refuses(ValueError, sv.spec_scan, **{**s, "b": s["b"][:, :, 0]})
    refuses(ValueError, sv.spec_scan, **{**s, "c": torch.zeros((2, 3, 2, 16))})
    refuses(ValueError, sv.spec_scan, **{**s, "c": torch.zeros((2, 3, 1, 32))[..., ::2]})
    refuses(TypeError, sv.spec_scan, **{**s, "a": s["a"].double()})
    refuses(ValueError, sv.spec_scan, **{**s, "a": s["a"][:7]})
    refuses(ValueError, sv.spec_scan, **s, skip=torch.zeros(7))
    refuses(ValueError, sv.spec_scan, **s, z=x[..., :7])
    refuses(TypeError, sv.spec_scan, **s, lens=torch.zeros(2))
    refuses(ValueError, sv.spec_scan, **s)                                       # on the host
    refuses(ValueError, sv.new_scan_workspace, 1, 1, 8, 12, "cpu")
    kv, i32 = torch.zeros((5, 2, 16, 64), dtype=torch.bfloat16), lambda *v: torch.tensor(v, dtype=torch.int32)
    cache = i32(0, 1, 2), i32(3, 3), torch.zeros((2, 3), dtype=torch.int32), kv, kv
    q = torch.zeros((2, 8, 64), dtype=torch.bfloat16)
    refuses(ValueError, sv.spec_attend_shared, q, i32(0, 2), i32(3, 3), *cache, max_tokens=1)
    refuses(ValueError, sv.spec_attend_shared, q, i32(0, 1, 2, 2), i32(3, 3, 3), *cache, max_tokens=1)
    refuses(TypeError, sv.spec_attend_shared, q, i32(0, 2).long(), i32(3), *cache, max_tokens=1)
    refuses(TypeError, sv.spec_attend_shared, q.float(), i32(0, 2), i32(3), *cache, max_tokens=1)
    refuses(ValueError, sv.spec_attend_shared, q[:, :5], i32(0, 2), i32(3), *cache, max_tokens=1)
    refuses(ValueError, sv.spec_attend_shared, q, i32(0, 2), i32(3), *cache, max_tokens=1)           # on the host
    refuses(ValueError, sv.new_attend_shared_workspace, 2, 2, 2, 4, 80, "cpu")
