"""Speculative decoding of a small hybrid model through the library's calls.

    python examples/verify_forward.py [--pool e4m3|bf16] [--rows 6] [--rounds 24]

The target has one attention layer over a paged cache and one gated linear
recurrence; the draft model is its output layer on a token's embedding alone.
Weights are random.  A prompt is read in one chunk (spec_cache_write, spec_attend,
spec_recur with lengths); each round then drafts k tokens (spec_draft_sample),
runs the target over the k + 1 tokens of every row (the same three calls, the
recurrence writing a state per token) and verifies them and commits the state of
the last accepted one (spec_verify_commit).  A rejected token's keys and values
stay in the cache, where the next round writes over them.

At the end the accepted tokens are read again as prompts: the states and the
cache that the rounds left must be those.  `fit_gates` trains a recurrence's
gates by spec_recur_backward.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from speculative_decoding_verify_07_gb300 import binding as sv  # noqa: E402


class Target:
    def __init__(self, vocab, width, heads, group, head_dim, dev):
        gen = torch.Generator(device=dev).manual_seed(7)

        def weight(*shape):
            w = torch.randn(shape, generator=gen, device=dev) * shape[0] ** -0.5
            return w.to(torch.bfloat16)

        self.vocab, self.width, self.heads, self.group, self.dim = vocab, width, heads, group, head_dim
        self.embed = (weight(vocab, width) * vocab ** 0.5).contiguous()
        self.qkv = weight(width, (group + 2) * heads * head_dim)
        self.merge = weight(group * heads * head_dim, width) * 0.5
        self.gates = weight(width, 2 * width) * 0.5
        self.head = weight(width, vocab)

    @staticmethod
    def norm(x):
        return torch.nn.functional.rms_norm(x, x.shape[-1:])


class Rows:
    """The serving state of a batch: paged cache, recurrent states, lengths."""

    def __init__(self, target, rows, most, pool, dev, page=16):
        pages = -(-most // page)
        shape = (rows * pages, target.heads, page, target.dim)
        dtype = torch.float8_e4m3fn if pool == "e4m3" else torch.bfloat16
        self.k, self.v = (torch.zeros(shape, dtype=torch.uint8 if pool == "e4m3" else dtype, device=dev).view(dtype) for _ in range(2))
        self.exps = tuple(torch.zeros(shape[:3], dtype=torch.uint8, device=dev) for _ in range(2)) if pool == "e4m3" else (None, None)
        self.table = torch.randperm(rows * pages, device=dev).to(torch.int32).view(rows, pages).contiguous()
        self.kv_len = torch.zeros(rows, dtype=torch.int32, device=dev)
        self.state = torch.zeros((1, rows, 1, 1, target.width), device=dev)
        self.slot = torch.arange(rows - 1, -1, -1, dtype=torch.int32, device=dev)
        self.flags = torch.zeros(rows, dtype=torch.int32, device=dev)
        self.attend_space = sv.new_attend_workspace(target.heads, target.group, target.dim, dev)
        self.recur_space = sv.new_recur_workspace(rows, most, target.width, dev)

    def cache(self, cu):
        return cu, self.kv_len, self.table, self.k, self.v, *self.exps


def forward(m, rows, tokens, lens, h=None, last=None):
    """Logits [B, T, V] of tokens [B, T], of which row r has lens[r]; keys, values go to the cache.  h: where the states
    of all tokens go; last: the cache of states that takes the last one."""
    B, T = tokens.shape
    inside = torch.arange(T, device=tokens.device)[None] < lens[:, None]
    cu = torch.nn.functional.pad(lens.cumsum(0), (1, 0)).to(torch.int32)
    rows.kv_len += lens
    x = m.embed[tokens.long()]
    heads, group, dim = m.heads, m.group, m.dim
    qkv = (m.norm(x)[inside] @ m.qkv).view(-1, (group + 2) * heads, dim)      # packed tokens, heads side by side
    q, k, v = qkv[:, :group * heads], qkv[:, group * heads:-heads], qkv[:, -heads:]
    sv.spec_cache_write(k, v, *rows.cache(cu), flags=rows.flags)
    a, _ = sv.spec_attend(q, *rows.cache(cu), max_tokens=T, flags=rows.flags, workspace=rows.attend_space)
    x = x.clone()
    x[inside] += a.flatten(1) @ m.merge
    g, y = (m.norm(x) @ m.gates).split(m.width, -1)
    g = -torch.nn.functional.softplus(g - 1)
    state = rows.state.view(B, m.width)
    h, _ = sv.spec_recur(g, y, state, rows.slot, lens, h=h, last=last, last_slot=None if last is None else rows.slot,
                         flags=rows.flags, workspace=rows.recur_space)
    return m.norm(x.float() + h).to(torch.bfloat16) @ m.head


def prefill(m, rows, prompts, lens):
    """Reads the prompts; their last token's logits."""
    logits = forward(m, rows, prompts, lens, last=rows.state.view(-1, m.width))
    return logits[torch.arange(len(lens), device=lens.device), lens.long() - 1]


def generate(pool="e4m3", batch=6, rounds=24, k=2, seed=11, dev="cuda"):
    """Returns what the rounds left and what reading the same tokens at once leaves, and tokens a round and row."""
    torch.manual_seed(seed)
    m = Target(vocab=2048, width=256, heads=2, group=4, head_dim=64, dev=dev)
    lens = torch.tensor([5 + 13 * r for r in range(batch)], dtype=torch.int32, device=dev)
    most = int(lens.max())
    room = most + (k + 1) * (rounds + 1)
    prompts = torch.randint(0, m.vocab, (batch, most), dtype=torch.int32, device=dev)
    params = sv.make_params([0.9] * batch, [40] * batch, [0.95] * batch, dev)
    rows = Rows(m, batch, room, pool, dev)
    first = sv.spec_draft_sample(prefill(m, rows, prompts, lens), params, seed, 0, with_q=False).tokens
    texts = [prompts[r, :lens[r]].tolist() for r in range(batch)]
    newest, emitted = first, 0
    verify_states = torch.empty((1, batch, k + 1, 1, 1, m.width), device=dev)
    each = torch.full((batch,), k + 1, dtype=torch.int32, device=dev)
    for step in range(rounds):
        fed, qs = [newest], []
        for j in range(k):
            logits = m.norm(m.embed[fed[-1].long()]) @ m.head
            d = sv.spec_draft_sample(logits.contiguous(), params, seed + 1 + step, j)
            fed.append(d.tokens)
            qs.append(d.q)
        tokens = torch.stack(fed, 1)
        logits = forward(m, rows, tokens, each, h=verify_states.view(batch, k + 1, m.width))
        out = sv.spec_verify_commit(logits.contiguous(), torch.stack(qs, 1).contiguous(), tokens[:, 1:].contiguous(), params,
                                    seed + 1000 + step, verify_states, None, rows.slot, rows.state, None)
        rows.kv_len += out.accept_len - (k + 1)           # the accepted tokens stay, the rest is written over
        took = out.accept_len.tolist()
        newest = out.tokens[torch.arange(batch, device=dev), out.accept_len.long() - 1].contiguous()
        for r in range(batch):
            texts[r] += tokens[r, :took[r]].tolist()      # what is now in the cache: the fed tokens that were accepted
        emitted += sum(took)
    assert not rows.flags.any(), rows.flags
    again = Rows(m, batch, room, pool, dev)
    lens = torch.tensor([len(t) for t in texts], dtype=torch.int32, device=dev)
    assert torch.equal(lens, rows.kv_len)
    longest = int(lens.max())
    padded = torch.tensor([t + [0] * (longest - len(t)) for t in texts], dtype=torch.int32, device=dev)
    prefill(m, again, padded, lens)
    cu = torch.nn.functional.pad(lens.cumsum(0), (1, 0)).to(torch.int32)
    kept, read = (sv.spec_cache_read(int(cu[-1]), *r.cache(cu)) for r in (rows, again))
    torch.cuda.synchronize()
    return dict(states=(rows.state.flatten(), again.state.flatten()), cache=(torch.stack(kept), torch.stack(read)),
                per_round=emitted / rounds / batch)


class Recurrence(torch.autograd.Function):
    @staticmethod
    def forward(ctx, g, x):
        h, _ = sv.spec_recur(g, x)
        ctx.save_for_backward(g, h)
        return h

    @staticmethod
    def backward(ctx, dh):
        g, h = ctx.saved_tensors
        dg, dx, _ = sv.spec_recur_backward(g, h, dh.to(g.dtype).contiguous())
        return dg, dx


def fit_gates(steps=60, dev="cuda"):
    """Learns the decays of a recurrence from its outputs; the loss at each step."""
    torch.manual_seed(3)
    B, T, D = 4, 512, 64
    x = torch.randn((B, T, D), device=dev)
    wanted = Recurrence.apply((-torch.linspace(0.02, 1.0, D, device=dev)).expand(B, T, D), x)
    rate = torch.full((D,), -1.0, device=dev, requires_grad=True)
    adam, losses = torch.optim.Adam([rate], lr=0.1), []
    for _ in range(steps):
        h = Recurrence.apply((-torch.exp(rate)).expand(B, T, D), x)
        loss = (h - wanted).square().mean()
        adam.zero_grad()
        loss.backward()
        adam.step()
        losses.append(loss.detach())
    return torch.stack(losses).tolist()


def main():
    p = argparse.ArgumentParser()
    p.add_argument("--pool", default="e4m3", choices=["e4m3", "bf16"])
    p.add_argument("--rows", type=int, default=6)
    p.add_argument("--rounds", type=int, default=24)
    a = p.parse_args()
    r = generate(a.pool, a.rows, a.rounds)
    for name in ("states", "cache"):
        left, read = (t.float() for t in r[name])
        print(f"{name}: rounds against one reading, relative difference {float((left - read).norm() / read.norm()):.2e}")
    print(f"tokens a row and round: {r['per_round']:.2f}")
    losses = fit_gates()
    print(f"gates: loss {losses[0]:.4f} -> {losses[-1]:.6f}")


if __name__ == "__main__":
    main()
