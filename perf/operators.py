"""The operators around a verify step, in plain form and through the library.

A speculative step runs a target forward over each row's k+1 new tokens before
spec_verify can judge them.  Its attention layers write the new keys and values
into a paged cache (spec_cache_write), read the cache through the page table
(spec_attend) and, where another engine wants them dense, read them back
(spec_cache_read); its recurrent layers scan the new tokens (spec_recur) and
leave one state a token for spec_commit; training the same layers runs that
scan over long sequences and back (spec_recur_backward).

Packed rows: row r's new tokens are cu[r] .. cu[r+1]-1 of the packed arrays,
kv_len[r] counts its cached tokens including the new ones, and its token at
position p lives in page table[r, p // page], slot p % page, of pools
[pages, heads, page, dim].  An e4m3 pool has one exponent byte e a (token,
head): a code c stands for c * 2^(e - 127).
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
E4M3 = torch.float8_e4m3fn


# ------------------------------------------------------------------ the cases

def listed():
    cache = dict(op="write", heads=8, dim=128, page=16, pool="e4m3", dtype="bf16")
    att = dict(op="attend", heads=8, group=4, dim=128, page=16, pool="e4m3")
    rec = dict(op="recur", dtype="bf16", h="f32", ragged=False, state=True, resets=False)
    return [
        # the cache write of one verify step: 64 rows of k + 1 = 3 tokens, a few microseconds of work
        dict(cache, name="write_verify_64x3", rows=64, tokens=3, ragged=False, past=400),
        # prompts of uneven lengths entering the cache at once
        dict(cache, name="write_prompts", rows=12, tokens=4096, ragged=True, past=0),
        # whole rows leaving the cache for another engine's dense layout
        dict(cache, op="read", name="read_rows", rows=16, tokens=6000, ragged=True, past=0),
        # one stream's plain decode step on a short context: latency
        dict(att, name="attend_one", rows=1, tokens=1, ragged=False, past=332, group=2, dim=64, pool="bf16"),
        # the verify step of 64 rows at k = 2 over contexts of uneven lengths, 8-bit cache
        dict(att, name="attend_verify_64x3", rows=64, tokens=3, ragged=False, past=12000),
        # 16 rows at k = 4 over long contexts, 16-bit cache, wide sharing of heads
        dict(att, name="attend_verify_16x5", rows=16, tokens=5, ragged=False, past=30000, heads=2, group=8, page=64,
             pool="bf16"),
        # chunks of long prompts behind what is cached of them
        dict(att, name="attend_chunk_2x2048", rows=2, tokens=2048, ragged=False, past=9000, page=32, pool="bf16"),
        # uneven chunks of odd sizes, 8-bit cache
        dict(att, name="attend_chunk_ragged", rows=5, tokens=1333, ragged=True, past=3001, dim=64, group=3),
        # the recurrent layer of the verify step: every position's state, as spec_commit takes it
        dict(rec, name="recur_verify_64x3", rows=64, tokens=3, dim=4096),
        # a long sequence alone: few rows, so its length has to be split
        dict(rec, name="recur_long", rows=1, tokens=65536, dim=2048, h="bf16", state=False),
        # a training step's layer, forward and backward, packed documents ending inside the rows
        dict(rec, op="train", name="recur_train", rows=4, tokens=8192, dim=2560, h="bf16", resets=True),
        # odd sizes, fp32, rows of uneven lengths
        dict(rec, op="train", name="recur_train_odd", rows=3, tokens=1021, dim=1337, dtype="f32", ragged=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["write", "read", "attend", "attend", "chunk", "recur", "train"])
    if op in ("write", "read"):
        c = dict(op=op, heads=rng.choice([1, 2, 3, 4, 8]), dim=rng.choice([64, 128]),
                 page=rng.choice([1, 16, 24, 32, 64, 128]), pool=rng.choice(["bf16", "e4m3", "e4m3"]),
                 dtype="bf16" if op == "read" else rng.choice(["bf16", "bf16", "f32"]), rows=_log(rng, 1, 200),
                 ragged=rng.random() < 0.6, past=rng.choice([0, _log(rng, 1, 500)]))
        c["tokens"] = _log(rng, 1, max(2, min(8192, 60000 // c["rows"])))
        return c
    if op in ("attend", "chunk"):
        c = dict(op="attend", heads=rng.choice([1, 2, 4, 8]), group=rng.choice([1, 2, 3, 4, 8, 16]),
                 dim=rng.choice([64, 128]), page=rng.choice([1, 16, 16, 24, 32, 64, 128]),
                 pool=rng.choice(["bf16", "e4m3"]), ragged=rng.random() < 0.5)
        if op == "attend":
            c["rows"] = _log(rng, 1, 128)
            c["tokens"] = rng.choice([1, 2, 3, 5, 9, 17])
            c["past"] = _log(rng, 1, min(60000, 350000 // c["rows"]))
        else:
            c["heads"], c["group"] = rng.choice([(1, 16), (2, 8), (4, 5), (4, 4), (8, 1), (8, 4)])
            c["rows"] = _log(rng, 1, 6)
            c["tokens"] = _log(rng, 32, 3000 // c["rows"])
            c["past"] = _log(rng, 1, 9000)
        return c
    c = dict(op=op, dim=_log(rng, 64, 4096), dtype=rng.choice(["bf16", "bf16", "f32"]), h=rng.choice(["bf16", "f32"]),
             ragged=rng.random() < 0.4, state=rng.random() < 0.6, resets=rng.random() < 0.3)
    if rng.random() < 0.6:
        c["dim"] = max(64, c["dim"] // 64 * 64)
    if op == "recur" and rng.random() < 0.4:
        c["rows"], c["tokens"] = _log(rng, 1, 256), rng.choice([1, 2, 3, 5, 17])
    else:
        c["rows"] = _log(rng, 1, 16)
        most = 36000000 if c["dtype"] == "f32" else 50000000
        c["tokens"] = _log(rng, 20, min(65536, most // (c["rows"] * c["dim"])))
    return c


# ---------------------------------------------------------------- their inputs

def _lengths(case, gen):
    """New tokens and cached tokens of each row, as lists."""
    n, rows = case["tokens"], case["rows"]
    if case["ragged"]:
        new = torch.randint(1, n + 1, (rows,), generator=gen).tolist()
        new[0] = n
    else:
        new = [n] * rows
    past = case["past"]
    if past > 1 and rows > 1:
        # what a batch has cached is spread from short to long
        cached = torch.randint(max(1, past // 16), past + 1, (rows,), generator=gen).tolist()
    else:
        cached = [past] * rows
    return new, [c + m for c, m in zip(cached, new)]


def _sizes(case):
    """The rows' lengths as the work counts them: those of seed 0."""
    return _lengths(case, torch.Generator().manual_seed(0))


def _lens(case):
    """How much of each row a recurrence scans: some rows may be empty."""
    n, rows = case["tokens"], case["rows"]
    if not case["ragged"]:
        return [n] * rows
    return [n] + torch.randint(0, n + 1, (rows - 1,), generator=torch.Generator().manual_seed(0)).tolist()


def _paged(case, seed):
    gen = torch.Generator().manual_seed(int(seed))
    new, total = _lengths(case, torch.Generator().manual_seed(0))
    page = case["page"]
    need = [(t + page - 1) // page for t in total]
    pages = sum(need) + 3
    order = torch.randperm(pages, generator=gen).tolist()
    table = torch.full((len(new), max(need)), -1, dtype=torch.int32)
    at = 0
    for r, m in enumerate(need):
        table[r, :m] = torch.tensor(order[at:at + m], dtype=torch.int32)
        at += m
    cu = torch.tensor([0] + new, dtype=torch.int32).cumsum(0, dtype=torch.int32)
    return {"cu": cu.to(DEV), "kv_len": torch.tensor(total, dtype=torch.int32, device=DEV), "table": table.to(DEV),
            "pages": pages, "tokens": sum(new), "max_tokens": max(new), "max_kv": max(total)}


def _quantised(x):
    """e4m3 codes and exponent bytes of vectors in the last dimension: the smallest power of two that brings the
    largest magnitude to 448 or less.  Scaling by it is exact; the code is the one rounding."""
    amax = x.float().abs().amax(-1)
    m, e = torch.frexp(amax)                       # amax = m 2^e, m in [0.5, 1); 448 = 0.875 * 2^9
    e = (e - 9 + (m > 0.875).to(e.dtype)).clamp(-126, 127)
    return torch.ldexp(x.float(), -e[..., None]).to(E4M3), (e + 127).to(torch.uint8)


def _pools(case, pages, gen, empty):
    shape = (pages, case["heads"], case["page"], case["dim"])
    made = {}
    for n in ("k", "v"):
        if empty:
            x = torch.zeros(shape, dtype=torch.bfloat16, device=DEV)
        else:
            x = torch.empty(shape, dtype=torch.bfloat16, device=DEV).normal_(generator=gen)
        if case["pool"] == "e4m3":
            made[n + "_pages"], made[n + "_exp"] = _quantised(x)
        else:
            made[n + "_pages"], made[n + "_exp"] = x, None
        del x
    return made


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(int(seed))
    s = {"case": case, "op": case["op"]}
    if case["op"] in ("write", "read", "attend"):
        s.update(_paged(case, seed))
        s.update(_pools(case, s["pages"], gen, case["op"] == "write"))
        shape = (s["tokens"], case["heads"], case["dim"])
        if case["op"] == "write":
            # keys and values of one token differ in size from head to head and from token to token
            size = torch.exp(torch.randn(shape[:2], device=DEV, generator=gen))[..., None]
            for n in ("k", "v"):
                s[n] = (torch.randn(shape, device=DEV, generator=gen) * size).to(DTYPES[case["dtype"]])
        if case["op"] == "attend":
            shape = (s["tokens"], case["heads"] * case["group"], case["dim"])
            # scores of a few units, so that a row's weight gathers on some of its keys
            s["q"] = (2.0 * torch.randn(shape, device=DEV, generator=gen)).to(torch.bfloat16)
        return s
    rows, n, dim, dt = case["rows"], case["tokens"], case["dim"], DTYPES[case["dtype"]]
    shape = (rows, n, dim)
    # decays from a half to a few thousandths a token, one kind of channel beside another
    pace = torch.rand((dim,), device=DEV, generator=gen) * 5.0 - 6.0
    g = -torch.exp(pace + 0.5 * torch.randn(shape, device=DEV, generator=gen))
    if case["resets"]:
        # documents begin here: nothing is carried over
        begins = torch.rand((rows, n), device=DEV, generator=gen) < 4.0 / max(n, 4)
        g[begins] = -math.inf
    s["g"] = g.to(dt)
    s["x"] = torch.randn(shape, device=DEV, generator=gen).to(dt)
    s["lens"] = torch.tensor(_lens(case), dtype=torch.int32, device=DEV) if case["ragged"] else None
    s["state"] = s["slot"] = None
    if case["state"]:
        slots = rows + 5
        s["state"] = torch.randn((slots, dim), device=DEV, generator=gen)
        s["slot"] = torch.randperm(slots, generator=torch.Generator().manual_seed(int(seed) + 1))[:rows].to(torch.int32).to(DEV)
    if case["op"] == "train":
        s["dh"] = torch.randn(shape, device=DEV, generator=gen).to(dt)
    return s


# ------------------------------------------------------------------ plain forms

def _rows_of(s):
    """The row and the position of each packed token."""
    token = torch.arange(s["tokens"], device=DEV)
    row = torch.searchsorted(s["cu"].long(), token, right=True) - 1
    cu, total = s["cu"].long(), s["kv_len"].long()
    return row, total[row] - (cu[row + 1] - token)


def _places(s, row, pos):
    page = s["case"]["page"]
    return s["table"].long()[row, pos // page], pos % page


def _values(pages, exps, page, slot):
    """What the cache holds at (page, slot) of equal shapes: [..., heads, dim] in 32 bits."""
    if exps is None:
        return pages[page, :, slot].float()
    codes = pages.view(torch.uint8)[page, :, slot].view(E4M3).float()
    return torch.ldexp(codes, exps[page, :, slot].int()[..., None] - 127)


def _plain_write(s):
    page, slot = _places(s, *_rows_of(s))
    for n in ("k", "v"):
        if s["case"]["pool"] == "e4m3":
            codes, exps = _quantised(s[n])
            s[n + "_pages"].view(torch.uint8)[page, :, slot] = codes.view(torch.uint8)
            s[n + "_exp"][page, :, slot] = exps
        else:
            s[n + "_pages"][page, :, slot] = s[n].to(torch.bfloat16)


def _plain_read(s):
    page, slot = _places(s, *_rows_of(s))
    return [_values(s[n + "_pages"], s[n + "_exp"], page, slot).to(torch.bfloat16) for n in ("k", "v")]


def _plain_attend(s):
    case = s["case"]
    heads, group, dim = case["heads"], case["group"], case["dim"]
    rows, most, width = case["rows"], s["max_tokens"], s["max_kv"]
    row, pos = _rows_of(s)
    col = torch.arange(s["tokens"], device=DEV) - s["cu"].long()[row]
    # every row's cache, dense up to the longest
    key = torch.arange(width, device=DEV).expand(rows, width)
    there = key < s["kv_len"].long()[:, None]
    page, slot = _places(s, torch.arange(rows, device=DEV)[:, None], key)
    page = torch.where(there, page, 0)
    k, v = (_values(s[n + "_pages"], s[n + "_exp"], page, slot).transpose(1, 2) for n in ("k", "v"))
    v = torch.where(there[:, None, :, None], v, 0.0)
    q = torch.zeros((rows, most, heads, group, dim), device=DEV)
    q[row, col] = s["q"].float().view(-1, heads, group, dim)
    last = torch.full((rows, most), -1, device=DEV)
    last[row, col] = pos
    q = q.permute(0, 2, 3, 1, 4).reshape(rows, heads, group * most, dim)
    score = q @ k.transpose(2, 3) * dim ** -0.5
    hidden = (key[:, None, :] > last[:, :, None]).repeat(1, group, 1)[:, None]
    score.masked_fill_(hidden, -math.inf)
    top = score.amax(-1, keepdim=True).clamp_min(torch.finfo(torch.float32).min)
    score.sub_(top).exp_()
    total = score.sum(-1, keepdim=True)
    out = (score @ v) / torch.where(total > 0, total, 1.0)
    lse = (total.log() + top)[..., 0]
    out = out.view(rows, heads, group, most, dim)[row, :, :, col]
    lse = lse.view(rows, heads, group, most)[row, :, :, col]
    return out.reshape(-1, heads * group, dim).to(torch.bfloat16), lse.reshape(-1, heads * group)


def _scan(a, b):
    """b_t + a_t (b_{t-1} + a_{t-1} (...)) along dimension 1, by doubling."""
    step = 1
    while step < b.shape[1]:
        b = torch.cat([b[:, :step], b[:, step:] + a[:, step:] * b[:, :-step]], 1)
        a = torch.cat([a[:, :step], a[:, step:] * a[:, :-step]], 1)
        step *= 2
    return b


def _within(s):
    """Which positions lie inside the rows' lengths, [rows, tokens, 1]; None where all do."""
    if s["lens"] is None:
        return None
    return (torch.arange(s["g"].shape[1], device=DEV)[None] < s["lens"][:, None])[..., None]


def _start(s):
    return None if s["state"] is None else s["state"][s["slot"].long()]


def _plain_recur(s):
    """All states in 32 bits, and the last one of each row."""
    a, b, inside, first = s["g"].float().exp(), s["x"].float(), _within(s), _start(s)
    if inside is not None:
        a, b = torch.where(inside, a, 1.0), torch.where(inside, b, 0.0)
    if first is not None:
        b = torch.cat([(b[:, 0] + a[:, 0] * first)[:, None], b[:, 1:]], 1)
    h = _scan(a, b)
    end = h[:, -1].clone()
    return (h if inside is None else torch.where(inside, h, 0.0)), end


def _plain_recur_backward(s, h):
    a, d, inside, first = s["g"].float().exp(), s["dh"].float(), _within(s), _start(s)
    if inside is not None:
        a, d = torch.where(inside, a, 1.0), torch.where(inside, d, 0.0)
    follows = torch.cat([a[:, 1:], torch.zeros_like(a[:, :1])], 1)        # the decay behind each position
    dx = _scan(follows.flip(1), d.flip(1)).flip(1)
    carried = a * dx
    before = torch.cat([torch.zeros_like(h[:, :1]) if first is None else first[:, None], h[:, :-1]], 1)
    dg = carried * before
    if inside is not None:
        dx, dg = torch.where(inside, dx, 0.0), torch.where(inside, dg, 0.0)
    return dg, dx, carried[:, 0]


def _plain(s):
    op = s["op"]
    if op == "write":
        _plain_write(s)
    elif op == "read":
        return _plain_read(s)
    elif op == "attend":
        return _plain_attend(s)
    else:
        h, end = _plain_recur(s)
        out = [h.to(DTYPES[s["case"]["h"]]), end]
        if op == "train":
            dg, dx, first = _plain_recur_backward(s, h)
            out += [dg.to(s["g"].dtype), dx.to(s["g"].dtype), first]
        return out
    return _written(s)


def _written(s):
    """The cache after a write: the values' codes and their exponents."""
    return [s[n] for n in ("k_pages", "v_pages", "k_exp", "v_exp") if s[n] is not None]


# ---------------------------------------------------------- through the library

def _library(s):
    from speculative_decoding_verify_07_gb300 import binding as sv
    op, case = s["op"], s["case"]
    if op in ("write", "read", "attend"):
        cache = (s["cu"], s["kv_len"], s["table"], s["k_pages"], s["v_pages"], s["k_exp"], s["v_exp"])
        if op == "write":
            sv.spec_cache_write(s["k"], s["v"], *cache)
            return _written(s)
        if op == "read":
            return list(sv.spec_cache_read(s["tokens"], *cache))
        if "workspace" not in s:
            s["workspace"] = sv.new_attend_workspace(case["heads"], case["group"], case["dim"], DEV)
        return sv.spec_attend(s["q"], *cache, max_tokens=s["max_tokens"], workspace=s["workspace"])
    if "workspace" not in s:
        s["workspace"] = sv.new_recur_workspace(case["rows"], case["tokens"], case["dim"], DEV)
    h, end = sv.spec_recur(s["g"], s["x"], s["state"], s["slot"], s["lens"], h_dtype=DTYPES[case["h"]],
                           workspace=s["workspace"])
    out = [h, end]
    if op == "train":
        out += sv.spec_recur_backward(s["g"], h, s["dh"], s["state"], s["slot"], s["lens"], workspace=s["workspace"])
    return out


def run(s):
    return _library(s) if own else _plain(s)


# ------------------------------------------------------------------------ work

def work(case):
    if case["op"] in ("write", "read", "attend"):
        new, total = _sizes(case)
        dim, heads = case["dim"], case["heads"]
        cell = 2 * dim if case["pool"] == "bf16" else dim + 1
        if case["op"] == "attend":
            hq = heads * case["group"]
            seen = sum(n * t - n * (n - 1) // 2 for n, t in zip(new, total))
            return {"bytes": 2 * heads * cell * sum(total) + sum(new) * hq * (4 * dim + 4), "flops": 4 * dim * hq * seen}
        each = 4 if case["dtype"] == "f32" else 2
        return {"bytes": 2 * heads * sum(new) * (cell + each * dim), "flops": 2 * heads * sum(new) * dim}
    every, scanned = case["rows"] * case["tokens"] * case["dim"], sum(_lens(case)) * case["dim"]
    g, h = (4 if case[n] == "f32" else 2 for n in ("dtype", "h"))
    states = case["rows"] * case["dim"] * 4 * (2 if case["state"] else 1)
    forward = scanned * 2 * g + every * h + states
    if case["op"] == "recur":
        return {"bytes": forward, "flops": 3 * scanned}
    return {"bytes": forward + scanned * (2 * g + h) + every * 2 * g + states, "flops": 8 * scanned}


# ------------------------------------------------- the definitions in 64 bits

def _exact_codes(x):
    """The nearest e4m3 value of x 2^-s, and s, from the format's own steps."""
    x = x.double()
    amax = x.abs().amax(-1, keepdim=True)
    s = torch.ceil(torch.log2(torch.where(amax > 0, amax, 1.0) / 448))
    s = torch.where(amax * torch.exp2(-s) > 448, s + 1, torch.where(amax * torch.exp2(1 - s) <= 448, s - 1, s))
    s = torch.where(amax > 0, s, -126.0).clamp(-126, 127)
    y = x * torch.exp2(-s)
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp_min(2.0 ** -6))) - 3)
    return torch.round(y / step) * step, s[..., 0]


def _exact_paged(case, s):
    rows = zip(s["cu"].tolist(), s["cu"].tolist()[1:], s["kv_len"].tolist(), s["table"].tolist())
    page, op = case["page"], case["op"]
    heads, dim = case["heads"], case["dim"]

    def cached(n, at, slot):
        pool, exps = s[n + "_pages"], s[n + "_exp"]
        if exps is None:
            return pool[at, :, slot].double()
        return pool.view(torch.uint8)[at, :, slot].view(E4M3).double() * torch.exp2(exps[at, :, slot].double() - 127)[..., None]

    if op == "write":
        out = [s[n + "_pages"].double() for n in ("k", "v")]
        exps = None
        if case["pool"] == "e4m3":
            exps = [s[n + "_exp"].clone() for n in ("k", "v")]
        for a, b, total, table in rows:
            p = torch.arange(total - (b - a), total)
            at, slot = torch.tensor(table)[p // page].to(DEV), (p % page).to(DEV)
            for i, n in enumerate(("k", "v")):
                if exps is None:
                    out[i][at, :, slot] = s[n][a:b].double()
                else:
                    out[i][at, :, slot], e = _exact_codes(s[n][a:b])
                    exps[i][at, :, slot] = (e + 127).to(torch.uint8)
        return out + (exps or [])
    if op == "read":
        out = [torch.empty((s["tokens"], heads, dim), dtype=torch.float64, device=DEV) for _ in range(2)]
    else:
        hq = heads * case["group"]
        out = [torch.empty((s["tokens"], hq, dim), dtype=torch.float64, device=DEV),
               torch.empty((s["tokens"], hq), dtype=torch.float64, device=DEV)]
    for a, b, total, table in rows:
        p = torch.arange(total - (b - a) if op == "read" else 0, total)
        at, slot = torch.tensor(table)[p // page].to(DEV), (p % page).to(DEV)
        k, v = cached("k", at, slot), cached("v", at, slot)
        if op == "read":
            out[0][a:b], out[1][a:b] = k, v
            continue
        late = torch.arange(total, device=DEV)[None] > torch.arange(total - (b - a), total, device=DEV)[:, None]
        for i in range(hq):
            w = s["q"][a:b, i].double() @ k[:, i // case["group"]].T / math.sqrt(dim)
            w = torch.where(late, -math.inf, w)
            lse = torch.logsumexp(w, 1)
            out[0][a:b, i] = torch.exp(w - lse[:, None]) @ v[:, i // case["group"]]
            out[1][a:b, i] = lse
    return out


def exact(case, seed):
    if work(case)["flops"] > 4e12 or case["rows"] * case["tokens"] * case["dim"] > 2e8:
        return None
    s = prepare(case, seed)
    if case["op"] in ("write", "read", "attend"):
        return _exact_paged(case, s)
    rows, n, dim = s["g"].shape
    lens = torch.full((rows,), n, device=DEV) if s["lens"] is None else s["lens"]
    state = torch.zeros((rows, dim), dtype=torch.float64, device=DEV)
    if s["state"] is not None:
        state = s["state"][s["slot"].long()].double()
    h = torch.empty((rows, n, dim), dtype=torch.float64, device=DEV)
    before = torch.empty_like(h)
    a = torch.exp(s["g"].double())
    for t in range(n):
        live = (t < lens)[:, None]
        before[:, t] = state
        state = torch.where(live, torch.addcmul(s["x"][:, t].double(), a[:, t], state), state)
        h[:, t] = torch.where(live, state, 0.0)
    out = [h, state]
    if case["op"] == "train":
        dg, dx = torch.empty_like(h), torch.empty_like(h)
        carry = torch.zeros((rows, dim), dtype=torch.float64, device=DEV)
        for t in reversed(range(n)):
            live = (t < lens)[:, None]
            lam = torch.where(live, s["dh"][:, t].double() + carry, 0.0)
            dx[:, t] = lam
            carry = torch.where(live, a[:, t] * lam, carry)
            dg[:, t] = torch.where(live, a[:, t] * lam * before[:, t], 0.0)
        out += [dg, dx, carry]
    return out
