"""fp64 definition of the attention operators (numpy): the norm and rotation
of queries and keys (by positions of one axis or several), attention with a sliding window and sinks, and its step
over a paged cache.  Test infrastructure; no code shared with the library.
"""
from __future__ import annotations

import numpy as np


def qk_norm_rope(x, positions, weight=None, eps=None, inv_freq=None, interleaved=False):
    """x [B,H,T,d], positions [B,T] -> (y, size): the operator's result and
    |a| + |b| of every channel's pair (|y| where it does not rotate), the
    scale of its rounding errors.  eps None: no norm."""
    x = np.asarray(x, np.float64)
    y = x
    if eps is not None:
        y = x / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps)
        if weight is not None:
            y = y * np.asarray(weight, np.float64)
    y = y.copy()
    size = np.abs(y)
    if inv_freq is not None:
        inv_freq = np.asarray(inv_freq, np.float64)
        half = len(inv_freq)
        for i in range(half):
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
            th = np.asarray(positions, np.float64)[:, None, :] * inv_freq[i]
            c, s = np.cos(th), np.sin(th)
            u, w = y[..., a].copy(), y[..., b].copy()
            y[..., a], y[..., b] = u * c - w * s, w * c + u * s
            size[..., a] = size[..., b] = np.abs(u) + np.abs(w)
    return y, size


def qk_norm_rope_axes(x, positions, axis, weight=None, eps=None, inv_freq=None, interleaved=False):
    """The same with positions [axes,B,T] and the axis of each pair [rot/2]."""
    x = np.asarray(x, np.float64)
    y, size = qk_norm_rope(x, np.zeros(np.asarray(positions).shape[1:]), weight, eps)
    if inv_freq is None:
        return y, size
    half = len(inv_freq)
    z, y = y, y.copy()
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        th = np.asarray(positions, np.float64)[axis[i]][:, None, :] * float(inv_freq[i])
        # the pair as one complex number, turned
        turned = (z[..., a] + 1j * z[..., b]) * np.exp(1j * th)
        y[..., a], y[..., b] = turned.real, turned.imag
        size[..., a] = size[..., b] = np.abs(z[..., a]) + np.abs(z[..., b])
    return y, size


def sees(p, j, klen, window, sinks):
    return (0 <= j) and (j < klen) and (j <= p) and ((j > p - window) or (j < sinks))


def row(q, k, v, scale):
    """One row over the keys it sees (k, v [n, d]): its output, the weighted
    sum of |v| and max_j scale sum_c |q_c k_jc| (scales of rounding errors)."""
    if len(k) == 0:
        z = np.zeros(v.shape[-1])
        return z, z, 0.0
    s = (k @ q) * scale
    m = np.max(s)
    if m == -np.inf:
        z = np.zeros(v.shape[-1])
        return z, z, 0.0
    with np.errstate(invalid="ignore"):
        w = np.exp(s - m)
        w = w / np.sum(w)
        return w @ v, w @ np.abs(v), float(np.max(np.abs(k) @ np.abs(q)) * abs(scale))


def window(q, k, v, window, sinks, scale, q_len=None, k_len=None):
    """q [B,Hq,Tq,d], k, v [B,Hk,Tk,d] -> (o, size, reach, written): output,
    the weighted sums of |v|, every row's score scale [B,Hq,Tq], and which
    rows are written [B,Tq]."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    B, Hq, Tq, d = q.shape
    Hk, Tk = k.shape[1:3]
    o, size = np.zeros(q.shape), np.zeros(q.shape)
    reach, written = np.zeros((B, Hq, Tq)), np.zeros((B, Tq), bool)
    for b in range(B):
        ql = Tq if q_len is None else int(q_len[b])
        kl = Tk if k_len is None else int(k_len[b])
        written[b, :ql] = True
        for i in range(ql):
            p = kl - ql + i
            # the range that the definition's inequalities leave
            lo = max(0, p - window + 1)
            keys = [j for j in range(0, min(sinks, lo))] + list(range(lo, min(p + 1, kl)))
            for h in range(Hq):
                g = h // (Hq // Hk)
                o[b, h, i], size[b, h, i], reach[b, h, i] = row(q[b, h, i], k[b, g, keys], v[b, g, keys], scale)
    return o, size, reach, written


def step(q, k_cache, v_cache, table, lens, window, sinks, scale):
    """q [N,Hq,d], pools [P,Hk,page,d], table [N,most], lens [N] -> (o, size,
    reach, written)."""
    q, k_cache, v_cache = (np.asarray(x, np.float64) for x in (q, k_cache, v_cache))
    N, Hq, d = q.shape
    Hk, page = k_cache.shape[1:3]
    o, size, reach = np.zeros(q.shape), np.zeros(q.shape), np.zeros((N, Hq))
    written = np.zeros(N, bool)
    for n in range(N):
        L = int(lens[n])
        written[n] = L >= 0
        keys = np.array([j for j in range(L) if sees(L - 1, j, L, window, sinks)], int)
        pages, rows = np.asarray(table)[n][keys // page], keys % page
        for h in range(Hq):
            g = h // (Hq // Hk)
            o[n, h], size[n, h], reach[n, h] = row(q[n, h], k_cache[pages, g, rows], v_cache[pages, g, rows], scale)
    return o, size, reach, written


def attention_bound(o, size, reach, keys, d, dtype_bits, weight_bits=None):
    """Elementwise bound on |result - o|.

    Rounding: the result once, at half a step u = 2^-dtype_bits of |o|; the
    weights to 2^-weight_bits where the product takes them in fewer bits, each
    moving the output by that part of size = sum_j w_j |v_j|.  fp32: a score is
    a sum of d products, off by (d + 4) 2^-23 reach; the exponential's argument
    (at most 2 reach) is rounded twice and its result is off by 2^-21; sums
    over `keys` values add keys 2^-24.  An error f of the weights, relative,
    moves numerator and denominator, so 2 f size."""
    f = (d + 4) * 2.0 ** -23 * reach + 2 * reach * 2.0 ** -23 + 2.0 ** -21 + (keys + 8) * 2.0 ** -24
    b = 2 * f[..., None] * size + 2.0 ** -dtype_bits * np.abs(o)
    if weight_bits is not None:
        b = b + 2 * 2.0 ** -weight_bits * size
    return b + 1e-37


def _maps(q, k, v, seen, scale):
    """q [T,d], k [J,d], v [J,c], seen [T,J] -> output, sizes and reach as in row(), for all rows."""
    used = seen.any(0)
    k, v = np.where(used[:, None], k, 0.0), np.where(used[:, None], v, 0.0)
    s = np.where(seen, (q @ k.T) * scale, -np.inf)
    m = s.max(-1, keepdims=True, initial=-np.inf)
    w = np.exp(s - np.where(np.isinf(m), 0.0, m))
    n = w.sum(-1, keepdims=True)
    w = w / np.where(n > 0, n, 1.0)
    reach = np.where(seen, np.abs(q) @ np.abs(k).T, 0.0).max(-1, initial=0.0) * abs(scale)
    return w @ v, w @ np.abs(v), reach


def diff_rows(q0, q1, k0, k1, v, seen, scale, lam, d, dtype_bits, weight_bits=None, weight=None, eps=None):
    """Rows of one pair of heads -> (o, bound), both [T,2d].  eps None: no norm.

    The bound: each map's row is off as attention_bound has it but for the
    result's rounding; the difference adds one rounding of each term.  The norm
    r = sqrt(mean y^2 + eps) moves by at most the root mean square e of the errors,
    so y / r by (err + |y| e / r) / (r - e); its own arithmetic adds (d + 8) 2^-24
    of the result, which is then rounded once."""
    keys = seen.shape[1]
    y, err = 0.0, 0.0
    for m, (q, k, factor) in enumerate(((q0, k0, 1.0), (q1, k1, lam))):
        a, size, reach = _maps(q, k, v, seen, scale)
        y = a if m == 0 else y - factor * a
        part = attention_bound(a, size, reach, keys, d, 24, weight_bits)
        err = part if m == 0 else err + abs(factor) * part
        err = err + 2.0 ** -23 * abs(factor) * np.abs(a)
    if eps is None:
        return y, err + 2.0 ** -dtype_bits * np.abs(y)
    r = np.sqrt(np.mean(y * y, -1, keepdims=True) + eps)
    e = np.sqrt(np.mean(err * err, -1, keepdims=True))
    none = ~(y != 0).any(-1, keepdims=True)
    with np.errstate(divide="ignore", invalid="ignore"):
        o = np.where(none, 0.0, y / r)
        off = np.where(e < r, (err + np.abs(y) * e / r) / (r - e), np.inf)
    w = 1.0 if weight is None else np.asarray(weight, np.float64)
    o = o * w
    seen_none = ~seen.any(-1)[:, None]
    return o, np.where(seen_none, 0.0, off * np.abs(w) + ((d + 8) * 2.0 ** -24 + 2.0 ** -dtype_bits) * np.abs(o) + 1e-37)


def diff(q, k, v, lam, window, sinks, scale, dtype_bits, weight_bits=None, weight=None, eps=None, q_len=None,
         k_len=None):
    """q [B,2H,Tq,d], k, v [B,2Hk,Tk,d] -> (o, bound, written [B,Tq])."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    B, H2, Tq, d = q.shape
    Hk2, Tk = k.shape[1:3]
    G = H2 // Hk2
    o, bound, written = np.zeros(q.shape), np.zeros(q.shape), np.zeros((B, Tq), bool)
    for b in range(B):
        ql = Tq if q_len is None else int(q_len[b])
        kl = Tk if k_len is None else int(k_len[b])
        written[b, :ql] = True
        p, j = kl - ql + np.arange(ql)[:, None], np.arange(Tk)
        seen = (j < kl) & (j <= p) & ((j > p - window) | (j < sinks))
        for h in range(H2 // 2):
            g = h // G
            y, e = diff_rows(q[b, 2 * h, :ql], q[b, 2 * h + 1, :ql], k[b, 2 * g], k[b, 2 * g + 1],
                             np.concatenate((v[b, 2 * g], v[b, 2 * g + 1]), -1), seen, scale, float(lam[h]), d,
                             dtype_bits, weight_bits, weight, eps)
            for half in range(2):
                o[b, 2 * h + half, :ql] = y[:, half * d:(half + 1) * d]
                bound[b, 2 * h + half, :ql] = e[:, half * d:(half + 1) * d]
    return o, bound, written


def diff_step(q, k_cache, v_cache, table, lens, lam, window, sinks, scale, dtype_bits, weight_bits=None, weight=None,
              eps=None):
    """q [N,2H,d], pools [P,2Hk,page,d] -> (o, bound, written [N])."""
    q, k_cache, v_cache = (np.asarray(x, np.float64) for x in (q, k_cache, v_cache))
    N, H2, d = q.shape
    Hk2, page = k_cache.shape[1:3]
    o, bound, written = np.zeros(q.shape), np.zeros(q.shape), np.zeros(N, bool)
    for n in range(N):
        L = int(lens[n])
        written[n] = L >= 0
        keys = np.array([j for j in range(L) if sees(L - 1, j, L, window, sinks)], int)
        where, rows = np.asarray(table)[n][keys // page], keys % page
        seen = np.ones((1, len(keys)), bool)
        for h in range(H2 // 2):
            g = h // (H2 // Hk2)
            k = [k_cache[where, 2 * g + m, rows] for m in range(2)]
            v = np.concatenate([v_cache[where, 2 * g + m, rows] for m in range(2)], -1)
            y, e = diff_rows(q[n, 2 * h][None], q[n, 2 * h + 1][None], *k, v, seen, scale, float(lam[h]), d, dtype_bits,
                             weight_bits, weight, eps)
            o[n, 2 * h:2 * h + 2], bound[n, 2 * h:2 * h + 2] = y.reshape(2, d), e.reshape(2, d)
    return o, bound, written


def step_prefix(q, k_cache, v_cache, prefix, prefix_len, table, lens, window, sinks, scale):
    """step() of sequences whose first prefix_len tokens are in the pages of
    `prefix`, their own lens[n] tokens behind them in those of table[n]."""
    q, k_cache, v_cache = (np.asarray(x, np.float64) for x in (q, k_cache, v_cache))
    N, Hq, d = q.shape
    Hk, page = k_cache.shape[1:3]
    o, size, reach = np.zeros(q.shape), np.zeros(q.shape), np.zeros((N, Hq))
    written = np.zeros(N, bool)
    for n in range(N):
        written[n] = lens[n] >= 0
        L = prefix_len + int(lens[n])
        if lens[n] < 0:
            continue
        keys = [j for j in range(L) if sees(L - 1, j, L, window, sinks)]
        at = [(prefix, j) if j < prefix_len else (table[n], j - prefix_len) for j in keys]
        pages = np.array([int(t[j // page]) for t, j in at], int)
        rows = np.array([j % page for _, j in at], int)
        for h in range(Hq):
            g = h // (Hq // Hk)
            o[n, h], size[n, h], reach[n, h] = row(q[n, h], k_cache[pages, g, rows], v_cache[pages, g, rows], scale)
    return o, size, reach, written
