"""Several samples of one prompt decoded speculatively by a hybrid model through the library's calls.

    python examples/verify_group.py [--pool e4m3|bf16] [--samples 6] [--rounds 12]

The target has one attention layer over a paged cache and one state space layer
(a short causal convolution and a selective scan); the draft model is its output
layer on a token's embedding alone.  Weights are random.  The prompt's whole pages
are read once, by one row; the samples share these pages and begin with the states
behind them, and read the rest of the prompt each for itself.  A round drafts k
tokens (spec_draft_sample), runs the target over the k + 1 tokens of every row
(spec_attend_shared; spec_conv and spec_scan with a state a token) and verifies them
and commits the states of the last accepted one (spec_verify_commit).

At the end one sample's text is read again by itself: the states that the rounds
left must be those.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from speculative_decoding_verify_07_gb300 import binding as sv  # noqa: E402


class Target:
    def __init__(self, vocab=2048, width=256, heads=2, group=4, dim=64, states=16, taps=4, dev="cuda"):
        gen = torch.Generator(device=dev).manual_seed(7)

        def weight(*shape):
            return (torch.randn(shape, generator=gen, device=dev) * shape[0] ** -0.5).to(torch.bfloat16)

        self.vocab, self.width, self.heads, self.group, self.dim, self.states = vocab, width, heads, group, dim, states
        self.embed = (weight(vocab, width) * vocab ** 0.5).contiguous()
        self.qkv = weight(width, (group + 2) * heads * dim)
        self.merge = weight(group * heads * dim, width) * 0.5
        self.inner = weight(width, 2 * width)                               # what is convolved, and its gate
        self.taps = torch.randn((taps, width), generator=gen, device=dev) * taps ** -0.5
        self.select = weight(width, width + 2 * states)                     # the steps, b and c
        self.a = -torch.arange(1, states + 1, device=dev).repeat(width, 1).float()
        step = torch.exp(torch.rand(width, generator=gen, device=dev) * 4.0 - 6.0)
        self.bias = step + torch.log(-torch.expm1(-step))                   # what softplus takes to the step
        self.skip = torch.ones(width, device=dev)
        self.head = weight(width, vocab)

    @staticmethod
    def norm(x):
        return torch.nn.functional.rms_norm(x, x.shape[-1:])


class Cache:
    """The serving state of `rows` rows: paged keys and values, the states of the other layer, lengths."""

    def __init__(self, m, rows, table, pages, page, pool, dev="cuda"):
        shape = (pages, m.heads, page, m.dim)
        dtype = torch.float8_e4m3fn if pool == "e4m3" else torch.bfloat16
        self.k, self.v = (torch.zeros(shape, dtype=torch.uint8 if pool == "e4m3" else dtype, device=dev).view(dtype) for _ in range(2))
        self.exps = tuple(torch.zeros(shape[:3], dtype=torch.uint8, device=dev) for _ in range(2)) if pool == "e4m3" else (None, None)
        self.table, self.kv_len = table, torch.zeros(rows, dtype=torch.int32, device=dev)
        # one layer's states, as spec_commit takes them
        self.rec = torch.zeros((1, rows, 1, m.width, m.states), device=dev)
        self.conv = torch.zeros((1, rows, len(m.taps) - 1, m.width), dtype=torch.bfloat16, device=dev)
        self.slot = torch.arange(rows - 1, -1, -1, dtype=torch.int32, device=dev)
        self.flags = torch.zeros(rows, dtype=torch.int32, device=dev)

    def pages(self, cu, rows):
        return cu, self.kv_len[rows], self.table[rows], self.k, self.v, *self.exps


def forward(m, cache, rows, tokens, common=None, states=None):
    """Logits [B, T, V] of tokens [B, T] of the cache's rows `rows` (a slice).  common: (shared_rows, shared_len), or None for
    rows of their own; states: where the states of all tokens go, (recurrent, convolution), or None: the cache has the last."""
    B, T = tokens.shape
    cu = torch.arange(0, B * T + 1, T, dtype=torch.int32, device=tokens.device)
    cache.kv_len[rows] += T
    flags, slot = cache.flags[rows], cache.slot[rows].contiguous()
    x = m.embed[tokens.long()]
    qkv = (m.norm(x) @ m.qkv).view(B * T, (m.group + 2) * m.heads, m.dim)
    q, k, v = qkv[:, :m.group * m.heads], qkv[:, m.group * m.heads:-m.heads], qkv[:, -m.heads:]
    pages = cache.pages(cu, rows)
    sv.spec_cache_write(k, v, *pages, flags=flags)
    if common is None:
        a, _ = sv.spec_attend(q, *pages, max_tokens=T, flags=flags)
    else:
        a, _ = sv.spec_attend_shared(q, *common, *pages, max_tokens=T, flags=flags)
    x = x + (a.flatten(1) @ m.merge).view(B, T, m.width)
    u, z = (m.norm(x) @ m.inner).split(m.width, -1)
    rec, conv = cache.rec[0, :, 0], cache.conv[0]
    keep = dict(last_slot=slot, flags=flags)
    u, _ = sv.spec_conv(u, m.taps, None, conv, slot, states=None if states is None else states[1], **(keep | dict(last=conv) if states is None else {}))
    dt, b, c = (u @ m.select).split([m.width, m.states, m.states], -1)
    y, _ = sv.spec_scan(u, dt, m.a, b[:, :, None], c[:, :, None], m.skip, z, m.bias, rec, slot, states=None if states is None else states[0],
                        **(keep | dict(last=rec) if states is None else {}))
    return m.norm((x + y).float()).to(torch.bfloat16) @ m.head


def generate(pool="bf16", samples=6, prompt_len=300, rounds=12, k=2, page=16, seed=11, dev="cuda"):
    """Returns the states that the rounds left of sample 0 and those of reading its text at once, and tokens a round and row."""
    torch.manual_seed(seed)
    m = Target(dev=dev)
    prompt = torch.randint(0, m.vocab, (1, prompt_len), dtype=torch.int32, device=dev)
    whole, room = prompt_len // page, -(-(prompt_len + (k + 1) * (rounds + 1)) // page)
    own = room - whole
    table = torch.cat([torch.arange(whole, device=dev).repeat(samples, 1),
                       whole + torch.randperm(samples * own, device=dev).view(samples, own)], 1).to(torch.int32).contiguous()
    cache = Cache(m, samples, table, whole + samples * own, page, pool)
    first = slice(0, 1)
    if whole:
        forward(m, cache, first, prompt[:, :whole * page])
        # the others begin behind the common pages
        cache.kv_len[:] = whole * page
        for states in (cache.rec, cache.conv):
            states[:] = states[:, cache.slot[:1].long()]
    everyone = slice(0, samples)
    common = (torch.tensor([0, samples], dtype=torch.int32, device=dev), torch.tensor([whole * page], dtype=torch.int32, device=dev))
    # the last token of the prompt is fed with the first round
    rest = prompt[:, whole * page:-1].repeat(samples, 1)
    if prompt_len % page == 0:
        raise ValueError("the prompt's last token must lie behind its whole pages")
    if rest.shape[1]:
        forward(m, cache, everyone, rest.contiguous(), common)
    params = sv.make_params([0.9] * samples, [40] * samples, [0.95] * samples, dev)
    newest = prompt[:, -1].repeat(samples).contiguous()
    texts = [prompt[0, :-1].tolist() for _ in range(samples)]
    verify_rec = torch.empty((1, samples, k + 1, 1, m.width, m.states), device=dev)
    verify_conv = torch.empty((1, samples, k + 1, len(m.taps) - 1, m.width), dtype=torch.bfloat16, device=dev)
    emitted = 0
    for step in range(rounds):
        fed, qs = [newest], []
        for j in range(k):
            d = sv.spec_draft_sample((m.norm(m.embed[fed[-1].long()]) @ m.head).contiguous(), params, seed + 1 + step, j)
            fed.append(d.tokens)
            qs.append(d.q)
        tokens = torch.stack(fed, 1)
        logits = forward(m, cache, everyone, tokens, common, (verify_rec.view(samples, k + 1, m.width, m.states), verify_conv[0]))
        out = sv.spec_verify_commit(logits.contiguous(), torch.stack(qs, 1).contiguous(), tokens[:, 1:].contiguous(), params,
                                    seed + 1000 + step, verify_rec, verify_conv, cache.slot, cache.rec, cache.conv)
        cache.kv_len += out.accept_len - (k + 1)          # the accepted tokens stay, the rest is written over
        took = out.accept_len.tolist()
        newest = out.tokens[torch.arange(samples, device=dev), out.accept_len.long() - 1].contiguous()
        for r in range(samples):
            texts[r] += tokens[r, :took[r]].tolist()
        emitted += sum(took)
    assert not cache.flags.any(), cache.flags
    assert cache.kv_len.tolist() == [len(t) for t in texts]
    again = Cache(m, 1, torch.arange(room, dtype=torch.int32, device=dev)[None].contiguous(), room, page, pool)
    forward(m, again, first, torch.tensor([texts[0]], dtype=torch.int32, device=dev))
    assert not again.flags.any(), again.flags
    slot = int(cache.slot[0])
    torch.cuda.synchronize()
    return dict(rec=(cache.rec[0, slot], again.rec[0, 0]), conv=(cache.conv[0, slot], again.conv[0, 0]), per_round=emitted / rounds / samples)


def main():
    p = argparse.ArgumentParser()
    p.add_argument("--pool", default="bf16", choices=["e4m3", "bf16"])
    p.add_argument("--samples", type=int, default=6)
    p.add_argument("--rounds", type=int, default=12)
    a = p.parse_args()
    r = generate(a.pool, a.samples, rounds=a.rounds)
    for name in ("rec", "conv"):
        left, read = (t.float() for t in r[name])
        print(f"{name}: rounds against one reading, relative difference {float((left - read).norm() / read.norm()):.2e}")
    print(f"tokens a row and round: {r['per_round']:.2f}")


if __name__ == "__main__":
    main()
