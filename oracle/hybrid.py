"""The mixers of hybrid targets in float64: the short causal convolution, the
selective scan, and which positions a group of rows has in common.

Plain loops over rows and tokens from the definitions; no code is shared with the
CUDA path.  Arrays are NumPy.
"""
import numpy as np


def silu(v):
    return v / (1.0 + np.exp(-v))


def conv(x, weight, bias, first, lens, gate):
    """(y, last, states, v, size) of y_t = act(bias + sum_i weight_i x_{t - W + 1 + i}).

    x [B, T, C], weight [W, C], first [B, W - 1, C] the inputs before each row; v is the sum before the gate and size the
    sum of its terms' magnitudes, which roundings scale with.  Zeros beyond lens."""
    x, weight, first = (np.asarray(a, np.float64) for a in (x, weight, first))
    B, T, C = x.shape
    K = len(weight) - 1
    bias = np.zeros(C) if bias is None else np.asarray(bias, np.float64)
    v, size, states = np.zeros((B, T, C)), np.zeros((B, T, C)), np.zeros((B, T, K, C))
    y, last = np.zeros((B, T, C)), np.zeros((B, K, C))
    for r in range(B):
        window = [first[r, i] for i in range(K)]
        for t in range(int(lens[r])):
            window.append(x[r, t])
            v[r, t] = bias + sum(w * s for w, s in zip(weight, window))
            size[r, t] = np.abs(bias) + sum(np.abs(w * s) for w, s in zip(weight, window))
            y[r, t] = silu(v[r, t]) if gate else v[r, t]
            window = window[1:]
            states[r, t] = window
        last[r] = window
    return y, last, states, v, size


def scan(x, dt, a, b, c, skip, z, dt_bias, first, lens, softplus):
    """(y, last, states, err) of the selective scan; err = (of y, of last, of states).

    x, dt, z [B, T, D], a [D, N], b, c [B, T, groups, N], first [B, D, N].  err counts roundings of float32, in half steps
    (2^-24 relative): of a step's delta up to 12 + |dt + bias|, so of delta x b up to that and 4; of a decay exp(g) up to
    6 + 24 |g|; of a state one; of the sum over N states N + 4 of its terms' magnitudes; of the gate 10 + 1.5 |z|."""
    x, dt, a, b, c, first = (np.asarray(v, np.float64) for v in (x, dt, a, b, c, first))
    B, T, D = x.shape
    N, groups = a.shape[1], b.shape[2]
    of = np.arange(D) // (D // groups)
    zero = np.zeros(D)
    skip, bias = (zero if v is None else np.asarray(v, np.float64) for v in (skip, dt_bias))
    y, states, last = np.zeros((B, T, D)), np.zeros((B, T, D, N)), np.array(first, np.float64)
    ey, es, el = np.zeros((B, T, D)), np.zeros((B, T, D, N)), np.zeros((B, D, N))
    for r in range(B):
        h, e = last[r], el[r]
        for t in range(int(lens[r])):
            raw = dt[r, t] + bias
            delta = np.logaddexp(0.0, raw) if softplus else raw
            g = delta[:, None] * a
            decay, put = np.exp(g), (delta * x[r, t])[:, None] * b[r, t][of]
            unsure = 16.0 + np.abs(raw)[:, None]
            e = decay * (e + (6.0 + (12.0 + unsure) * np.abs(g)) * np.abs(h)) + unsure * np.abs(put)
            h = decay * h + put
            e = e + np.abs(h)
            states[r, t], es[r, t] = h, e
            terms = c[r, t][of] * h
            v = terms.sum(1) + skip * x[r, t]
            ev = (np.abs(c[r, t][of]) * e).sum(1) + (N + 4) * (np.abs(terms).sum(1) + np.abs(skip * x[r, t]))
            if z is not None:
                s = silu(np.asarray(z[r, t], np.float64))
                ev = np.abs(s) * (ev + (10.0 + 1.5 * np.abs(z[r, t])) * np.abs(v))
                v = v * s
            y[r, t], ey[r, t] = v, ev
        last[r], el[r] = h, e
    return y, last, states, (ey, el, es)


def shared_positions(table, shared_rows, shared_len, cu, kv_len, pages, page_size):
    """Where each row finds each of its positions, [B, positions]: page * page_size + slot, or -1 without a valid page.

    What a group of two rows or more with new tokens has in common, in whole tiles of 128, is found through its first
    row's table.  With the cache seen as pages of one position this is the table that spec_attend would be given."""
    B, n = len(kv_len), table.shape[1] * page_size
    i, slot = np.divmod(np.arange(n), page_size)
    own = np.where((table >= 0) & (table < pages), table, -1)[:, i]
    own = np.where(own >= 0, own * page_size + slot, -1)
    out, rows = own.copy(), np.asarray(shared_rows)
    if (rows < 0).any() or (rows > B).any() or (np.diff(rows) < 0).any():
        return out
    for g in range(len(shared_len)):
        mine = [r for r in range(rows[g], rows[g + 1]) if cu[r + 1] > cu[r]]
        if len(mine) < 2:
            continue
        common = min([int(shared_len[g]), n] + [max(0, int(kv_len[r])) - int(cu[r + 1] - cu[r]) for r in mine])
        common = max(0, common) // 128 * 128
        out[mine, :common] = own[rows[g], :common]
    return out


def one_a_page(values):
    """[pages, heads, page_size, D] as pages of one position."""
    pages, heads, page_size, dim = values.shape
    return values.transpose(0, 2, 1, 3).reshape(pages * page_size, heads, 1, dim)
