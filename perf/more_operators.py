"""The mixers of a hybrid target's verify step, in plain form and through the library.

A hybrid target has state space layers beside its attention layers.  Their tokens
pass a short causal convolution (spec_conv) and a selective scan (spec_scan), for
a prompt over its whole length, in a verify step over k + 1 tokens a row, each
leaving the state that spec_commit may gather.  Where several samples of a prompt
are decoded side by side, their attention (spec_attend_shared) reads the cache of
what they have in common once for all of them.

Rows of the convolution and the scan are [rows, tokens, channels] with a length
each.  Those of the attention are packed: row r's new tokens are cu[r] ..
cu[r+1]-1, kv_len[r] counts its cached tokens including the new ones, and its token
at position p lives in page table[r, p // page], slot p % page, of pools
[pages, heads, page, dim].  An e4m3 pool has one exponent byte e a (token, head): a
code c stands for c * 2^(e - 127).  Rows shared_rows[g] .. shared_rows[g+1]-1 have
their first shared_len[g] positions in common.
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
E4M3 = torch.float8_e4m3fn


# ------------------------------------------------------------------ the cases

def listed():
    conv = dict(op="conv", width=4, dtype="bf16", ragged=False, state=True, states=False, silu=True, bias=True)
    scan = dict(op="scan", n=16, groups=1, dtype="bf16", ragged=False, state=True, states=False, gate=True, softplus=True)
    att = dict(op="shared", heads=8, group=4, dim=128, page=16, pool="bf16")
    return [
        # the convolution of a verify step: 64 rows of k + 1 = 3 tokens, a state a token for the commit
        dict(conv, name="conv_verify_64x3", rows=64, tokens=3, dim=4096, states=True),
        # prompts of uneven lengths
        dict(conv, name="conv_prompts", rows=4, tokens=8192, dim=4096, ragged=True, state=False),
        # odd sizes, fp32, another width
        dict(conv, name="conv_odd", rows=3, tokens=1021, dim=1337, dtype="f32", width=3, ragged=True),
        # one stream's plain decode step: latency
        dict(scan, name="scan_one", rows=1, tokens=1, dim=2048),
        # the scan of a verify step: every position's state, as spec_commit takes it
        dict(scan, name="scan_verify_64x3", rows=64, tokens=3, dim=4096, states=True),
        # prompts read at once
        dict(scan, name="scan_prompts", rows=4, tokens=2048, dim=4096, state=False),
        # a long sequence alone: few channels for the whole device
        dict(scan, name="scan_long", rows=1, tokens=32768, dim=2048),
        # odd sizes, fp32, two groups of B and C, rows of uneven lengths, no gate
        dict(scan, name="scan_odd", rows=3, tokens=1021, dim=1338, n=8, groups=2, dtype="f32", ragged=True, gate=False),
        # two samples of one short prompt, plain decode: latency
        dict(att, name="shared_two", prompts=1, samples=2, tokens=1, prefix=700, rest=20, dim=64, group=2),
        # the verify step of 64 samples of one long prompt at k = 2
        dict(att, name="shared_verify_64x3", prompts=1, samples=64, tokens=3, prefix=16000, rest=1000),
        # 16 prompts of 8 samples each, plain decode over an 8-bit cache
        dict(att, name="shared_groups_16x8", prompts=16, samples=8, tokens=1, prefix=6001, rest=600, pool="e4m3"),
        # questions of uneven lengths behind one long system prompt, read at once
        dict(att, name="shared_chunks", prompts=1, samples=6, tokens=500, prefix=12345, rest=0, page=64, heads=4),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["conv", "scan", "scan", "shared", "shared"])
    if op == "shared":
        c = dict(op=op, dim=rng.choice([64, 128]), page=rng.choice([1, 16, 16, 24, 32, 64, 128]),
                 pool=rng.choice(["bf16", "bf16", "e4m3"]), prompts=_log(rng, 1, 16))
        c["heads"], c["group"] = rng.choice([(1, 8), (2, 8), (4, 5), (4, 4), (8, 1), (8, 4), (2, 3)])
        c["samples"] = _log(rng, 1, min(64, 192 // c["prompts"]))
        rows = c["prompts"] * c["samples"]
        c["tokens"] = rng.choice([1, 1, 2, 3, 5, 9, _log(rng, 17, max(18, 1500 // rows))])
        c["prefix"] = _log(rng, 1, min(30000, 200000 // c["prompts"], 6000000 // (rows * c["tokens"])))
        c["rest"] = rng.choice([0, _log(rng, 1, min(4000, 60000 // rows))])
        return c
    c = dict(op=op, dim=_log(rng, 64, 4096), dtype=rng.choice(["bf16", "bf16", "f32"]), ragged=rng.random() < 0.4,
             state=rng.random() < 0.6, states=False)
    if rng.random() < 0.6:
        c["dim"] = max(64, c["dim"] // 64 * 64)
    if op == "conv":
        c.update(width=rng.choice([2, 3, 4, 4, 5, 8]), silu=rng.random() < 0.7, bias=rng.random() < 0.7)
        most = 30000000 if c["dtype"] == "f32" else 60000000
    else:
        c.update(n=rng.choice([8, 16, 16, 32, 64]), groups=rng.choice([1, 1, 2]), gate=rng.random() < 0.6,
                 softplus=rng.random() < 0.7)
        c["dim"] -= c["dim"] % c["groups"]
        most = 500000000 // c["n"]
    if rng.random() < 0.4:
        c["rows"], c["tokens"] = _log(rng, 1, 128), rng.choice([1, 2, 3, 5, 9])
        c["states"] = rng.random() < 0.5
        if op == "scan":
            c["rows"] = max(1, min(c["rows"], 25000000 // (c["n"] * c["dim"] * c["tokens"])))
    else:
        c["rows"] = _log(rng, 1, 16)
        c["tokens"] = _log(rng, 20, max(21, min(32768, most // (c["rows"] * c["dim"]))))
    return c


# ---------------------------------------------------------------- their inputs

def _lens(case):
    """How much of each row is there: some rows may be empty."""
    n, rows = case["tokens"], case["rows"]
    if not case["ragged"]:
        return [n] * rows
    return [n] + torch.randint(0, n + 1, (rows - 1,), generator=torch.Generator().manual_seed(0)).tolist()


def _lengths(case):
    """New tokens and cached tokens of each row of the attention."""
    gen, rows, n = torch.Generator().manual_seed(0), case["prompts"] * case["samples"], case["tokens"]
    new = [n] * rows
    if n > 16:          # chunks of prompts are uneven
        new = torch.randint(1, n + 1, (rows,), generator=gen).tolist()
    rest = torch.randint(0, case["rest"] + 1, (rows,), generator=gen).tolist()
    return new, [case["prefix"] + a + b for a, b in zip(rest, new)]


def _quantised(x):
    """e4m3 codes and exponent bytes of vectors in the last dimension, under the smallest fitting power of two."""
    amax = x.float().abs().amax(-1)
    m, e = torch.frexp(amax)                       # amax = m 2^e, m in [0.5, 1); 448 = 0.875 * 2^9
    e = (e - 9 + (m > 0.875).to(e.dtype)).clamp(-126, 127)
    return torch.ldexp(x.float(), -e[..., None]).to(E4M3), (e + 127).to(torch.uint8)


def _prepare_shared(case, seed, gen):
    new, total = _lengths(case)
    page, samples, prefix = case["page"], case["samples"], case["prefix"]
    common = prefix // page                        # whole pages that the samples share; a page begun is each one's own
    need = [-(-t // page) for t in total]
    pages = case["prompts"] * common + sum(m - common for m in need) + 3
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(int(seed))).tolist()
    table = torch.full((len(new), max(need)), -1, dtype=torch.int32)
    at, copies = 0, []
    for p in range(case["prompts"]):
        both = order[at:at + common]
        at += common
        for r in range(p * samples, (p + 1) * samples):
            rest = order[at:at + need[r] - common]
            at += len(rest)
            table[r, :need[r]] = torch.tensor(both + rest, dtype=torch.int32)
            if prefix % page and r > p * samples:
                copies.append((int(table[p * samples, common]), rest[0]))
    x = {}
    for n in ("k", "v"):
        pool = torch.empty((pages, case["heads"], page, case["dim"]), dtype=torch.bfloat16, device=DEV).normal_(generator=gen)
        if copies:
            src, dst = (torch.tensor(c, device=DEV) for c in zip(*copies))
            pool[dst, :, :prefix % page] = pool[src, :, :prefix % page]
        x[n + "_pages"], x[n + "_exp"] = _quantised(pool) if case["pool"] == "e4m3" else (pool, None)
    x.update(new=new, total=total, tokens=sum(new), table=table.to(DEV),
             cu=torch.tensor([0] + new, dtype=torch.int32).cumsum(0, dtype=torch.int32).to(DEV),
             kv_len=torch.tensor(total, dtype=torch.int32, device=DEV),
             shared_rows=torch.arange(0, len(new) + 1, samples, dtype=torch.int32, device=DEV),
             shared_len=torch.full((case["prompts"],), prefix, dtype=torch.int32, device=DEV))
    # scores of a few units, so that a row's weight gathers on some of its keys
    x["q"] = (2.0 * torch.randn((x["tokens"], case["heads"] * case["group"], case["dim"]), device=DEV, generator=gen)).to(torch.bfloat16)
    return x


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(int(seed))
    s = {"case": case, "op": case["op"]}
    if case["op"] == "shared":
        s.update(_prepare_shared(case, seed, gen))
        return s
    rows, n, dim, dt = case["rows"], case["tokens"], case["dim"], DTYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(shape, device=DEV, generator=gen)

    s["x"] = normal(rows, n, dim).to(dt)
    s["lens"] = torch.tensor(_lens(case), dtype=torch.int32, device=DEV) if case["ragged"] else None
    s["state"] = s["slot"] = s["states"] = None
    slots = rows + 5
    if case["state"]:
        s["slot"] = torch.randperm(slots, generator=torch.Generator().manual_seed(int(seed) + 1))[:rows].to(torch.int32).to(DEV)
    if case["op"] == "conv":
        k = case["width"] - 1
        s["weight"] = normal(k + 1, dim) * (k + 1) ** -0.5
        s["bias"] = 0.5 * normal(dim) if case["bias"] else None
        if case["state"]:
            s["state"] = normal(slots, k, dim).to(dt)
        if case["states"]:
            s["states"] = torch.empty((rows, n, k, dim), dtype=dt, device=DEV)
        return s
    N, G = case["n"], case["groups"]
    # B and C are columns of one projection, as a model computes them
    both = normal(rows, n, G, 2, N).to(dt)
    s["b"], s["c"] = both[:, :, :, 0], both[:, :, :, 1]
    # decays spread around -1 .. -N, steps around 0.001 .. 0.1 a channel
    s["a"] = -torch.arange(1, N + 1, device=DEV) * torch.exp(0.1 * normal(dim, N))
    step = torch.exp(torch.rand((dim,), device=DEV, generator=gen) * math.log(100.0) + math.log(0.001))
    if case["softplus"]:
        s["dt"] = (0.5 * normal(rows, n, dim)).to(dt)
        s["dt_bias"] = step + torch.log(-torch.expm1(-step))        # what softplus takes to the step
    else:
        s["dt"] = (step * torch.exp(0.5 * normal(rows, n, dim))).to(dt)
        s["dt_bias"] = None
    s["skip"] = normal(dim)
    s["z"] = normal(rows, n, dim).to(dt) if case["gate"] else None
    if case["state"]:
        s["state"] = normal(slots, dim, N)
    if case["states"]:
        s["states"] = torch.empty((rows, n, dim, N), device=DEV)
    return s


# ------------------------------------------------------------------ plain forms

def _inside(s, n):
    """Which positions lie inside the rows' lengths, [rows, tokens, 1]."""
    lens = s["lens"]
    if lens is None:
        return None
    return (torch.arange(n, device=DEV)[None] < lens[:, None])[..., None]


def _plain_conv(s):
    x, w, case = s["x"].float(), s["weight"], s["case"]
    rows, n, dim = x.shape
    k = case["width"] - 1
    start = torch.zeros((rows, k, dim), device=DEV) if s["state"] is None else s["state"][s["slot"].long()].float()
    padded = torch.cat([start, x], 1)
    y = sum(padded[:, i:i + n] * w[i] for i in range(k + 1))
    if s["bias"] is not None:
        y = y + s["bias"]
    if case["silu"]:
        y = y / (1.0 + torch.exp(-y))
    inside, dt = _inside(s, n), s["x"].dtype
    if inside is not None:
        y = torch.where(inside, y, 0.0)
    lens = torch.full((rows,), n, device=DEV) if s["lens"] is None else s["lens"].long()
    last = padded[torch.arange(rows, device=DEV)[:, None], lens[:, None] + torch.arange(k, device=DEV)]
    out = [y.to(dt), last.to(dt)]
    if s["states"] is not None:
        states = torch.stack([padded[:, 1 + i:1 + i + n] for i in range(k)], 2)
        if inside is not None:
            states = torch.where(inside[..., None], states, 0.0)
        out.append(states.to(dt))
    return out


def _doubled(a, b):
    """b_t + a_t (b_{t-1} + a_{t-1} (...)) along dimension 1, by doubling, and the products of the a."""
    step = 1
    while step < b.shape[1]:
        b = torch.cat([b[:, :step], b[:, step:] + a[:, step:] * b[:, :-step]], 1)
        a = torch.cat([a[:, :step], a[:, step:] * a[:, :-step]], 1)
        step *= 2
    return a, b


def _plain_scan(s):
    case = s["case"]
    x, delta = s["x"].float(), s["dt"].float()
    rows, n, dim = x.shape
    if s["dt_bias"] is not None:
        delta = delta + s["dt_bias"]
    if case["softplus"]:
        delta = delta.clamp_min(0) + torch.log1p(torch.exp(-delta.abs()))
    inside = _inside(s, n)
    if inside is not None:
        delta = torch.where(inside, delta, 0.0)
    b, c = (s[v].float().repeat_interleave(dim // case["groups"], 2) for v in ("b", "c")) if case["groups"] > 1 else \
        (s[v].float() for v in ("b", "c"))                          # [rows, tokens, dim or 1, n]
    h = torch.zeros((rows, dim, case["n"]), device=DEV) if s["state"] is None else s["state"][s["slot"].long()]
    y = torch.empty_like(x)
    piece = max(1, min(n, 2 ** 27 // (rows * dim * case["n"])))     # tokens at a time, for the memory that states take
    for t in range(0, n, piece):
        e = min(n, t + piece)
        d = delta[:, t:e, :, None]
        keep, put = _doubled(torch.exp(d * s["a"]), d * b[:, t:e] * x[:, t:e, :, None])
        states = put + keep * h[:, None]
        y[:, t:e] = (states * c[:, t:e]).sum(-1)
        h = states[:, -1]
        if s["states"] is not None:
            s["states"][:, t:e] = states
    y = y + s["skip"] * x
    if s["z"] is not None:
        z = s["z"].float()
        y = y * (z / (1.0 + torch.exp(-z)))
    if inside is not None:
        y = torch.where(inside, y, 0.0)
    out = [y.to(s["x"].dtype), h.clone()]
    if s["states"] is not None:
        if inside is not None:
            s["states"].masked_fill_(~inside[..., None], 0.0)
        out.append(s["states"])
    return out


def _cached(s, page, slot):
    """Keys and values at (page, slot) of equal shapes: [..., heads, dim] in 32 bits."""
    both = []
    for n in ("k", "v"):
        pool, exps = s[n + "_pages"], s[n + "_exp"]
        if exps is None:
            both.append(pool[page, :, slot].float())
        else:
            codes = pool.view(torch.uint8)[page, :, slot].view(E4M3).float()
            both.append(torch.ldexp(codes, exps[page, :, slot].int()[..., None] - 127))
    return both


def _plain_shared(s):
    case = s["case"]
    heads, group, dim, page, prefix, samples = (case[n] for n in ("heads", "group", "dim", "page", "prefix", "samples"))
    outs, lses, at = [], [], 0
    table, new, total = s["table"].long(), s["new"], s["total"]
    for p in range(case["prompts"]):
        rows = range(p * samples, (p + 1) * samples)
        count, most = sum(new[r] for r in rows), max(new[r] for r in rows)
        width = max(total[r] for r in rows) - prefix
        # queries in order, and by row, padded
        q = s["q"][at:at + count].float().view(count, heads, group, dim)
        cu = s["cu"][rows[0]:rows[-1] + 1].long()
        token = torch.arange(at, at + count, device=DEV)
        row = torch.searchsorted(cu, token, right=True) - 1
        col = token - cu[row]
        at += count
        pos = torch.arange(prefix, device=DEV)
        k, v = _cached(s, table[rows[0], pos // page], pos % page)                  # [prefix, heads, dim]
        qh = q.permute(1, 0, 2, 3).reshape(heads, count * group, dim) * dim ** -0.5
        first = (qh @ k.permute(1, 2, 0)).view(heads, count, group, prefix)
        # each row's own rest, padded to the longest
        own_pos = prefix + torch.arange(width, device=DEV)
        lengths = s["kv_len"][rows[0]:rows[-1] + 1].long()
        there = own_pos[None] < lengths[:, None]
        ids = torch.where(there, table[rows[0]:rows[-1] + 1][:, own_pos // page], 0)
        ko, vo = (t.transpose(1, 2) for t in _cached(s, ids, (own_pos % page).expand(samples, width)))   # [rows, heads, width, dim]
        vo = torch.where(there[:, None, :, None], vo, 0.0)
        qo = torch.zeros((samples, most, heads, group, dim), device=DEV)
        qo[row, col] = q * dim ** -0.5
        qo = qo.permute(0, 2, 3, 1, 4).reshape(samples, heads, group * most, dim)
        second = (qo @ ko.transpose(2, 3)).view(samples, heads, group, most, width)
        second = second[row, :, :, col].permute(1, 0, 2, 3)                         # [heads, tokens, group, width]
        last = lengths[row] - s["cu"][rows[0] + 1:rows[-1] + 2].long()[row] + token  # each token's position
        second.masked_fill_((own_pos[None] > last[:, None])[None, :, None], -math.inf)
        top = torch.maximum(first.amax(-1), second.amax(-1))
        first.sub_(top[..., None]).exp_()
        second.sub_(top[..., None]).exp_()
        sums = first.sum(-1) + second.sum(-1)
        out = (first.view(heads, count * group, prefix) @ v.transpose(0, 1)).view(heads, count, group, dim)
        wo = torch.zeros((samples, most, heads, group, width), device=DEV)
        wo[row, col] = second.permute(1, 0, 2, 3)
        wo = wo.permute(0, 2, 3, 1, 4).reshape(samples, heads, group * most, width)
        rest = (wo @ vo).view(samples, heads, group, most, dim)[row, :, :, col].permute(1, 0, 2, 3)
        outs.append(((out + rest) / sums[..., None]).permute(1, 0, 2, 3).reshape(count, heads * group, dim))
        lses.append((sums.log() + top).permute(1, 0, 2).reshape(count, heads * group))
    return [torch.cat(outs).to(torch.bfloat16), torch.cat(lses)]


# ---------------------------------------------------------- through the library

def _library(s):
    from speculative_decoding_verify_07_gb300 import binding as sv
    case = s["case"]
    if s["op"] == "conv":
        y, last = sv.spec_conv(s["x"], s["weight"], s["bias"], s["state"], s["slot"], s["lens"], silu=case["silu"],
                               states=s["states"])
    elif s["op"] == "scan":
        if "workspace" not in s:
            s["workspace"] = sv.new_scan_workspace(case["rows"], case["tokens"], case["dim"], case["n"], DEV)
        y, last = sv.spec_scan(s["x"], s["dt"], s["a"], s["b"], s["c"], s["skip"], s["z"], s["dt_bias"], s["state"], s["slot"],
                               s["lens"], softplus=case["softplus"], states=s["states"], workspace=s["workspace"])
    else:
        if "workspace" not in s:
            s["workspace"] = sv.new_attend_shared_workspace(s["tokens"], len(s["new"]), case["heads"], case["group"], case["dim"], DEV)
        return list(sv.spec_attend_shared(s["q"], s["shared_rows"], s["shared_len"], s["cu"], s["kv_len"], s["table"], s["k_pages"],
                                          s["v_pages"], s["k_exp"], s["v_exp"], max_tokens=max(s["new"]), workspace=s["workspace"]))
    return [y, last] if s["states"] is None else [y, last, s["states"]]


def run(s):
    if own:
        return _library(s)
    return {"conv": _plain_conv, "scan": _plain_scan, "shared": _plain_shared}[s["op"]](s)


# ------------------------------------------------------------------------ work

def work(case):
    if case["op"] == "shared":
        new, total = _lengths(case)
        dim, hq, prefix = case["dim"], case["heads"] * case["group"], case["prefix"]
        cell = 2 * dim if case["pool"] == "bf16" else dim + 1
        positions = case["prompts"] * prefix + sum(t - prefix for t in total)
        seen = sum(n * t - n * (n - 1) // 2 for n, t in zip(new, total))
        return {"bytes": 2 * case["heads"] * cell * positions + sum(new) * hq * (4 * dim + 4), "flops": 4 * dim * hq * seen}
    rows, n, dim = case["rows"], case["tokens"], case["dim"]
    each, there, every = 4 if case["dtype"] == "f32" else 2, sum(_lens(case)), rows * n
    if case["op"] == "conv":
        k = case["width"] - 1
        kept = rows * k * dim * (2 if case["state"] else 1) + (every * k * dim if case["states"] else 0)
        return {"bytes": each * (dim * (there + every) + kept) + 4 * dim * (k + 2),
                "flops": there * dim * (2 * case["width"] + (4 if case["silu"] else 0))}
    N = case["n"]
    kept = rows * dim * N * (2 if case["state"] else 1) + (every * dim * N if case["states"] else 0)
    return {"bytes": each * (dim * (there * (3 if case["gate"] else 2) + every) + 2 * there * N * case["groups"]) + 4 * (kept + dim * (N + 2)),
            "flops": there * dim * (7 * N + 8)}


# ------------------------------------------------- the definitions in 64 bits

def _exact_shared(case, s):
    heads, group, dim, page, samples = (case[n] for n in ("heads", "group", "dim", "page", "samples"))
    out = torch.empty((s["tokens"], heads * group, dim), dtype=torch.float64, device=DEV)
    lse = torch.empty((s["tokens"], heads * group), dtype=torch.float64, device=DEV)
    table, at = s["table"].cpu(), 0
    for r, (n, total) in enumerate(zip(s["new"], s["total"])):
        p = torch.arange(total)
        whose = torch.where(p < case["prefix"], r // samples * samples, r)
        pages, slots = table[whose, p // page].long().to(DEV), (p % page).to(DEV)
        kv = []
        for name in ("k", "v"):
            pool, exps = s[name + "_pages"], s[name + "_exp"]
            if exps is None:
                kv.append(pool[pages, :, slots].double())
            else:
                scale = torch.exp2(exps[pages, :, slots].double() - 127)
                kv.append(pool.view(torch.uint8)[pages, :, slots].view(E4M3).double() * scale[..., None])
        late = torch.arange(total, device=DEV)[None] > torch.arange(total - n, total, device=DEV)[:, None]
        for i in range(heads * group):
            w = s["q"][at:at + n, i].double() @ kv[0][:, i // group].T / math.sqrt(dim)
            w = torch.where(late, -math.inf, w)
            total_log = torch.logsumexp(w, 1)
            out[at:at + n, i] = torch.exp(w - total_log[:, None]) @ kv[1][:, i // group]
            lse[at:at + n, i] = total_log
        at += n
    return [out, lse]


def _exact_conv(case, s):
    x, w = s["x"].double(), s["weight"].double()
    rows, n, dim = x.shape
    k = case["width"] - 1
    lens = _lens(case)
    y, last = torch.zeros_like(x), torch.zeros((rows, k, dim), dtype=torch.float64, device=DEV)
    states = torch.zeros((rows, n, k, dim), dtype=torch.float64, device=DEV) if case["states"] else None
    for r in range(rows):
        before = torch.zeros((k, dim), dtype=torch.float64, device=DEV) if s["state"] is None else s["state"][int(s["slot"][r])].double()
        seen = torch.cat([before, x[r, :lens[r]]])
        v = torch.einsum("tci,ic->tc", seen.unfold(0, k + 1, 1), w) if lens[r] else x[r, :0]
        if s["bias"] is not None:
            v = v + s["bias"].double()
        y[r, :lens[r]] = v * torch.sigmoid(v) if case["silu"] else v
        last[r] = seen[len(seen) - k:]
        if states is not None and lens[r]:
            states[r, :lens[r]] = seen[1:].unfold(0, k, 1).transpose(1, 2)
    return [y, last] + ([states] if states is not None else [])


def _exact_scan(case, s):
    rows, n, dim = s["x"].shape
    each = dim // case["groups"]
    a = s["a"].double()
    h = torch.zeros((rows, dim, case["n"]), dtype=torch.float64, device=DEV)
    if s["state"] is not None:
        h = s["state"][s["slot"].long()].double()
    lens = torch.tensor(_lens(case), device=DEV)
    y = torch.zeros((rows, n, dim), dtype=torch.float64, device=DEV)
    states = torch.zeros((rows, n, dim, case["n"]), dtype=torch.float64, device=DEV) if case["states"] else None
    of_channel = torch.arange(dim, device=DEV) // each
    for t in range(n):
        live = t < lens
        x, d = s["x"][:, t].double(), s["dt"][:, t].double()
        if s["dt_bias"] is not None:
            d = d + s["dt_bias"].double()
        if case["softplus"]:
            d = torch.logaddexp(d, torch.zeros_like(d))
        b, c = s["b"][:, t].double()[:, of_channel], s["c"][:, t].double()[:, of_channel]
        now = torch.exp(d[..., None] * a) * h + (d * x)[..., None] * b
        h = torch.where(live[:, None, None], now, h)
        v = torch.einsum("rdn,rdn->rd", h, c) + s["skip"].double() * x
        if s["z"] is not None:
            z = s["z"][:, t].double()
            v = v * z * torch.sigmoid(z)
        y[:, t] = torch.where(live[:, None], v, 0.0)
        if states is not None:
            states[:, t] = torch.where(live[:, None, None], h, 0.0)
    return [y, h] + ([states] if states is not None else [])


def exact(case, seed):
    if case["op"] == "shared":
        # (so that its 64-bit products take seconds)
        return None if work(case)["flops"] > 3e12 else _exact_shared(case, prepare(case, seed))
    if case["op"] == "scan" and case["rows"] * case["tokens"] * case["dim"] * case["n"] > 3e9:
        return None
    s = prepare(case, seed)
    return _exact_conv(case, s) if case["op"] == "conv" else _exact_scan(case, s)
