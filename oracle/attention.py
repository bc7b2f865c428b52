"""fp64 definition of the attention operators (numpy): the norm and rotation
of queries and keys, attention with a sliding window and sinks, and its step
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
