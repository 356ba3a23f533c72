"""The forward's sequence mixers in float64: the e4m3 cache, attention over a
paged cache, the gated linear recurrence and its gradients.

Plain loops over rows and tokens from the definitions; no code is shared with
the CUDA path.  Arrays are NumPy; a paged cache is given as the values it
holds ([pages, heads, page_size, head_dim] float64, see `cache_values`).
"""
import numpy as np

F_NAN = 8
F_BAD_IDX = 128

# every finite e4m3 magnitude, by code: 2^-6 m/8 below code 8, then 2^(e-7) (1 + m/8)
_E4M3 = np.array([(c & 7) / 8 * 2.0 ** -6 if c < 8 else 2.0 ** ((c >> 3) - 7) * (1 + (c & 7) / 8) for c in range(127)])


def e4m3_value(codes):
    """The values of e4m3 codes (uint8)."""
    codes = np.asarray(codes, np.uint8)
    mag = np.append(_E4M3, np.nan)[codes & 0x7F]
    return np.where(codes & 0x80, -mag, mag)


def quantise(x):
    """(codes, exponent bytes, bad) of vectors in the last dimension."""
    x = np.asarray(x, np.float64)
    bad = ~np.isfinite(x).all(-1)
    x = np.where(bad[..., None], 0.0, x)
    amax = np.abs(x).max(-1)
    s = np.full(amax.shape, -126)
    for i in np.ndindex(amax.shape):
        while s[i] < 127 and amax[i] > 448.0 * 2.0 ** float(s[i]):
            s[i] += 1
    y = np.abs(x) * 2.0 ** -s[..., None].astype(np.float64)
    # nearest code; a tie goes to the even one
    hi = np.searchsorted(_E4M3, y).clip(0, 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = y - _E4M3[lo], _E4M3[hi] - y
    code = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    code = code.astype(np.uint8) | np.where(np.signbit(x), 0x80, 0).astype(np.uint8)
    code = np.where(bad[..., None], 0, code).astype(np.uint8)
    return code, np.where(bad, 255, s + 127).astype(np.uint8), bad


def cache_values(codes, exps):
    """What an e4m3 cache holds."""
    exps = np.asarray(exps).astype(np.int64)
    scale = np.where(exps == 255, np.nan, 2.0 ** (np.maximum(exps, 1) - 127.0))
    return e4m3_value(codes) * scale[..., None]


def places(cu, kv_len, table, pages, page_size):
    """(row, token, position, page or -1, slot) of every packed token."""
    out = []
    for r in range(len(kv_len)):
        for t in range(cu[r], cu[r + 1]):
            p = int(kv_len[r]) - int(cu[r + 1] - t)
            page = slot = -1
            if p >= 0:
                i, slot = divmod(p, page_size)
                if i < table.shape[1] and 0 <= table[r, i] < pages:
                    page = int(table[r, i])
            out.append((r, t, p, page, slot))
    return out


def _row_cache(r, n, table, k_values, v_values):
    """The row's first n positions, dense: keys, values [n, heads, D], and which positions have a page."""
    pages, _, page_size, _ = k_values.shape
    i, slot = np.divmod(np.arange(n), page_size)
    page = np.append(table[r], -1)[np.minimum(i, table.shape[1])]
    there = (page >= 0) & (page < pages)
    page = np.where(there, page, 0)
    return k_values[page, :, slot], v_values[page, :, slot], there


def attend(q, cu, kv_len, table, k_values, v_values, scale):
    """(out, lse, flags, size) of causal attention of new tokens over a paged
    cache; size is sum_j softmax_j |v_j|, what roundings of the weights scale with."""
    q = np.asarray(q, np.float64)
    N, hq, D = q.shape
    pages, heads, page_size, _ = k_values.shape
    out, lse, size = np.zeros((N, hq, D)), np.full((N, hq), -np.inf), np.zeros((N, hq, D))
    flags = np.zeros(len(kv_len), np.uint32)
    for r in range(len(kv_len)):
        for t in range(cu[r], cu[r + 1]):
            p = int(kv_len[r]) - int(cu[r + 1] - t)
            if p < 0:
                continue
            k, v, there = _row_cache(r, p + 1, table, k_values, v_values)
            if not there.all():
                flags[r] |= F_BAD_IDX
                k, v = k[there], v[there]
            if not len(k):
                continue
            for h in range(hq):
                hk = h // (hq // heads)
                with np.errstate(invalid="ignore"):
                    s = k[:, hk] @ q[t, h] * scale
                    top = s.max()
                    w = np.exp(s - (0.0 if np.isneginf(top) else top))
                    if w.sum() == 0.0:
                        continue
                    out[t, h] = w @ v[:, hk] / w.sum()
                    size[t, h] = w @ np.abs(v[:, hk]) / w.sum()
                    lse[t, h] = np.log(w.sum()) + top
    return out, lse, flags, size


def recur(g, x, first, lens):
    """(h, last) of h_t = exp(g_t) h_{t-1} + x_t; first [B, D]; zeros beyond lens."""
    g, x = np.asarray(g, np.float64), np.asarray(x, np.float64)
    h, last = np.zeros_like(g), np.array(first, np.float64)
    for r in range(g.shape[0]):
        for t in range(int(lens[r])):
            last[r] = np.exp(g[r, t]) * last[r] + x[r, t]
            h[r, t] = last[r]
    return h, last


def recur_backward(g, h, dh, first, lens, d_last):
    """(dg, dx, d_first) of recur, h being what it returned."""
    g, dh = np.asarray(g, np.float64), np.asarray(dh, np.float64)
    dg, dx, carry = np.zeros_like(g), np.zeros_like(g), np.array(d_last, np.float64)
    for r in range(g.shape[0]):
        for t in reversed(range(int(lens[r]))):
            dx[r, t] = dh[r, t] + carry[r]
            carry[r] = np.exp(g[r, t]) * dx[r, t]
            dg[r, t] = carry[r] * (h[r, t - 1] if t else first[r])
    return dg, dx, carry
