"""Cases that measure further attention operators: the rotation by positions of
several axes (with the write into a paged cache), the paged step of a batch
that shares a long prefix, and differential attention over whole sequences and
for single tokens.

``own`` false: plain torch; true: this repository's entry points.
"""
import math

import numpy as np
import torch

own = False

NO_WINDOW = 1 << 30
EPS = 1e-6


def _dev():
    return torch.device("cuda" if torch.cuda.is_available() else "cpu")


def _dt(case):
    return torch.float32 if case["dtype"] == "f32" else torch.bfloat16


def listed():
    return [
        # one decode step of a 64-sequence batch of a model that takes video: time, height and width, into the pages
        dict(name="axes_step", op="axes", dtype="bf16", B=64, T=1, Hq=32, Hk=8, d=128, rot=128, axes=3,
             interleaved=False, far=30000, page=64, append=True, ragged=False),
        # two video prompts at the sizes of the gated-delta prefill workload, into the pages
        dict(name="axes_video", op="axes", dtype="bf16", B=2, T=16384, Hq=16, Hk=4, d=128, rot=128, axes=3,
             interleaved=False, far=0, page=64, append=True, ragged=False),
        # padded images of odd sizes in fp32: height and width, neighbouring channels, half of them turned, no cache
        dict(name="axes_image_odd", op="axes", dtype="f32", B=3, T=777, Hq=6, Hk=2, d=64, rot=32, axes=2,
             interleaved=True, far=0, page=16, append=False, ragged=True),
        # a few requests on one system prompt: latency
        dict(name="prefix_few", op="prefix", dtype="bf16", N=4, Hq=32, Hk=8, d=128, P=2048, len_lo=1, len_hi=64,
             page=64, window=NO_WINDOW, sinks=0),
        # a serving batch on one long document
        dict(name="prefix_batch", op="prefix", dtype="bf16", N=128, Hq=32, Hk=8, d=128, P=16384, len_lo=100,
             len_hi=1024, page=64, window=NO_WINDOW, sinks=0),
        # fp32, a prefix that ends inside a page, a window that some rows have left behind, sinks in the prefix
        dict(name="prefix_f32_window", op="prefix", dtype="f32", N=33, Hq=8, Hk=4, d=64, P=1501, len_lo=1, len_hi=2000,
             page=16, window=1024, sinks=4),
        # short padded prompts: latency
        dict(name="diff_short", op="diff", dtype="bf16", B=4, H=4, Hk=2, Tq=173, Tk=173, d=64, window=NO_WINDOW,
             sinks=0, ragged=True, norm=True),
        # one long prompt, pairs of heads that share keys
        dict(name="diff_long", op="diff", dtype="bf16", B=1, H=8, Hk=4, Tq=8192, Tk=8192, d=64, window=NO_WINDOW,
             sinks=0, ragged=False, norm=True),
        # two prompts, wide heads (values of 256 channels), keys of their own
        dict(name="diff_wide", op="diff", dtype="bf16", B=2, H=8, Hk=8, Tq=4096, Tk=4096, d=128, window=NO_WINDOW,
             sinks=0, ragged=False, norm=True),
        # a later piece of padded prompts in fp32 with a window, odd sizes, no norm
        dict(name="diff_f32_piece", op="diff", dtype="f32", B=2, H=4, Hk=2, Tq=350, Tk=1501, d=64, window=300,
             sinks=3, ragged=True, norm=False),
        # one sequence being answered: latency
        dict(name="diff_step_one", op="diff_step", dtype="bf16", N=1, H=16, Hk=4, d=64, len_lo=1200, len_hi=1200,
             page=64, window=NO_WINDOW, sinks=0, norm=True),
        # a serving batch of very different lengths
        dict(name="diff_step_batch", op="diff_step", dtype="bf16", N=64, H=16, Hk=4, d=128, len_lo=500, len_hi=8192,
             page=64, window=NO_WINDOW, sinks=0, norm=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["axes", "prefix", "diff", "diff_step"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    d = rng.choice([32, 64, 128])
    Hk = rng.choice([1, 2, 3, 4, 8])
    group = rng.choice([1, 2, 3, 4, 8])
    wide = 2 if dtype == "f32" else 1
    window = NO_WINDOW if rng.random() < 0.5 else _log(rng, 1, 4096)
    sinks = rng.choice([0, 1, 4, 5, 64])
    page = rng.choice([16, 32, 64, 128])
    if op == "axes":
        Hq = Hk * group
        B = _log(rng, 1, 64)
        T = _log(rng, 1, max(1, min(16384, (2 * 16384 * 20 * 128) // (B * (Hq + Hk) * d * wide))))
        return dict(op=op, dtype=dtype, B=B, T=T, Hq=Hq, Hk=Hk, d=d, rot=rng.choice([d, d, d // 2]),
                    axes=rng.choice([1, 2, 3, 4]), interleaved=rng.random() < 0.5,
                    far=rng.choice([0, 5000, 1000000]), page=page, append=rng.random() < 0.5,
                    ragged=rng.random() < 0.4)
    if op == "prefix":
        Hq = Hk * group
        N = _log(rng, 1, 128)
        # fp32 products cost many times those of bf16: smaller prefixes
        most = (128 * 32 * 16384 * 128) // (N * Hq * d) // (16 if dtype == "f32" else 1)
        P = _log(rng, 1, max(1, min(65536, most)))
        hi = _log(rng, 1, max(1, min(8192, (128 * 1024 * 8 * 128) // (N * Hk * d * wide))))
        return dict(op=op, dtype=dtype, N=N, Hq=Hq, Hk=Hk, d=d, P=P, len_lo=max(1, hi // rng.choice([1, 2, 16])),
                    len_hi=hi, page=page, window=window, sinks=sinks)
    if op == "diff":
        H = Hk * rng.choice([1, 2, 3, 4])
        B = _log(rng, 1, 8)
        Tk = _log(rng, 1, 8192 if dtype == "bf16" else 1024)
        most = 8 * 8192 * 8192 * 64 // (1 if dtype == "bf16" else 16)
        while B > 1 and B * H * Tk * Tk * d > most:
            B -= 1
        while Tk > 1 and B * H * Tk * Tk * d > most:
            Tk -= max(1, Tk // 16)
        Tq = Tk if rng.random() < 0.6 else _log(rng, 1, Tk)
        return dict(op=op, dtype=dtype, B=B, H=H, Hk=Hk, Tq=Tq, Tk=Tk, d=d, window=window, sinks=sinks,
                    ragged=rng.random() < 0.5, norm=rng.random() < 0.7)
    H = Hk * rng.choice([1, 2, 3, 4])
    N = _log(rng, 1, 64)
    hi = _log(rng, 1, max(1, min(65536, (64 * 4096 * 4 * 128) // (N * Hk * d * wide))))
    return dict(op=op, dtype=dtype, N=N, H=H, Hk=Hk, d=d, len_lo=max(1, hi // rng.choice([1, 2, 16])), len_hi=hi,
                page=page, window=window, sinks=sinks, norm=rng.random() < 0.7)


# ------------------------------------------------------------------ inputs

def _lengths(case, seed):
    """The lengths of a step's sequences, drawn from the seed; the longest is there."""
    r = np.random.RandomState(seed % (1 << 31))
    lens = r.randint(case["len_lo"], case["len_hi"] + 1, case["N"])
    lens[r.randint(case["N"])] = case["len_hi"]
    return lens.astype(np.int32)


def _pages(r, lens, page):
    """A table [N, most] of distinct pages in no order, and the number of pages of the pool."""
    need = -(-np.asarray(lens) // page)
    most, total = max(1, int(need.max())), int(need.sum()) + 3
    order = r.permutation(total).astype(np.int32)
    table = np.zeros((len(need), most), np.int32)
    at = 0
    for n, c in enumerate(need):
        table[n, :c] = order[at:at + c]
        at += c
    return table, total


def _grid(r, T, axes, far):
    """Positions [axes, T] as a patched prompt has them: the last axis runs fastest, the first on from `far`."""
    side = max(1, int(round(T ** (1.0 / axes))) + int(r.randint(0, 3)))
    t = np.arange(T)
    pos = [(t // side ** (axes - 1 - a)) % (side if a else 1 << 30) for a in range(axes)]
    pos[0] = pos[0] + far
    return np.stack(pos)


def prepare(case, seed):
    dev, dt = _dev(), _dt(case)
    g = torch.Generator(dev)
    g.manual_seed(int(seed) * 7919 + 17)
    r = np.random.RandomState((int(seed) * 31 + 5) % (1 << 31))

    def normal(*shape, std=1.0, dtype=dt):
        return (torch.randn(*shape, generator=g, device=dev, dtype=torch.float32) * std).to(dtype)

    def ints(x):
        return torch.from_numpy(np.ascontiguousarray(x).astype(np.int32)).to(dev)

    s = dict(case=case)
    d, op = case["d"], case["op"]
    if op == "axes":
        B, T, Hq, Hk, A = case["B"], case["T"], case["Hq"], case["Hk"], case["axes"]
        # one projection's output, tokens first: q, k and v are views of it
        x = normal(B, T, Hq + 2 * Hk, d)
        s["q"], s["k"], s["v"] = (x[:, :, a:b].transpose(1, 2) for a, b in ((0, Hq), (Hq, Hq + Hk), (Hq + Hk, Hq + 2 * Hk)))
        s["qw"] = 1 + normal(d, std=0.1, dtype=torch.float32)
        s["kw"] = 1 + normal(d, std=0.1, dtype=torch.float32)
        half = case["rot"] // 2
        s["inv_freq"] = 10000.0 ** (-torch.arange(half, dtype=torch.float64, device=dev) / half)
        # the pairs in runs, one for each axis; the last axis takes what is left
        s["axis"] = ints(np.minimum(np.arange(half) * A // half, A - 1))
        first = r.randint(case["far"] // 2, case["far"] + 1, B)
        s["positions"] = ints(np.stack([_grid(r, T, A, f) for f in first], 1))
        # a token's row in its sequence differs from its positions; behind a prompt's end there is padding
        place = np.tile(np.arange(T), (B, 1)) + r.randint(0, 100, (B, 1)) * case["append"]
        if case["ragged"]:
            place[np.arange(T) >= r.randint(0, T + 1, (B, 1))] = -1
        s["places"] = ints(place)
        s["q_out"] = torch.zeros(B, Hq, T, d, dtype=dt, device=dev)
        s["k_out"] = torch.zeros(B, Hk, T, d, dtype=dt, device=dev)
        if case["append"]:
            table, total = _pages(r, np.full(B, T + 100), case["page"])
            s["table"] = ints(table)
            s["k_cache"] = torch.zeros(total, Hk, case["page"], d, dtype=dt, device=dev)
            s["v_cache"] = torch.zeros(total, Hk, case["page"], d, dtype=dt, device=dev)
    elif op == "prefix":
        N, Hq, Hk, page = case["N"], case["Hq"], case["Hk"], case["page"]
        lens = _lengths(case, int(seed))
        # the prefix is one more sequence of the pool
        table, total = _pages(r, np.concatenate((lens, [case["P"]])), page)
        s["prefix"] = ints(table[N, :-(-case["P"] // page)])
        s["table"], s["lens"] = ints(table[:N, :-(-int(lens.max()) // page)]), ints(lens)
        s["q"] = normal(N, Hq, d)
        s["k_cache"], s["v_cache"] = normal(total, Hk, page, d), normal(total, Hk, page, d)
    elif op == "diff":
        B, H, Hk, Tq, Tk = (case[n] for n in ("B", "H", "Hk", "Tq", "Tk"))
        # normed queries and keys in the library's layout, values as the projection leaves them
        s["q"], s["k"] = normal(B, 2 * H, Tq, d), normal(B, 2 * Hk, Tk, d)
        s["v"] = normal(B, Tk, 2 * Hk, d).transpose(1, 2)
        s["q_len"] = s["k_len"] = None
        if case["ragged"]:
            ql = r.randint(0 if B > 1 else 1, Tq + 1, B)
            ql[0] = Tq
            kl = np.minimum(ql + r.randint(0, Tk - Tq + 1, B), Tk)
            s["q_len"], s["k_len"] = ints(ql), ints(kl)
        # the heads of a token side by side, as the next projection reads them
        s["o"] = torch.zeros(B, Tq, 2 * H, d, dtype=dt, device=dev).transpose(1, 2)
    else:
        N, H, Hk, page = case["N"], case["H"], case["Hk"], case["page"]
        lens = _lengths(case, int(seed))
        table, total = _pages(r, lens, page)
        s["q"] = normal(N, 2 * H, d)
        s["k_cache"], s["v_cache"] = normal(total, 2 * Hk, page, d), normal(total, 2 * Hk, page, d)
        s["table"], s["lens"] = ints(table), ints(lens)
    if op in ("diff", "diff_step"):
        s["lam"] = torch.rand(case["H"], generator=g, device=dev) * 0.6 + 0.2
        s["weight"] = 0.4 * (1 + normal(2 * d, std=0.1, dtype=torch.float32)) if case["norm"] else None
    return s


# ------------------------------------------------------------- the operators

def _axes_plain(x, w, s):
    """x [B,H,T,d] -> 32 bits; angles in 64."""
    y = x.float()
    y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS) * w
    rot = s["case"]["rot"]
    p = s["positions"].double()[s["axis"].long()]            # [rot/2, B, T]
    th = p.permute(1, 2, 0)[:, None] * s["inv_freq"]
    c, n = torch.cos(th).float(), torch.sin(th).float()
    z, rest = y[..., :rot], y[..., rot:]
    if s["case"]["interleaved"]:
        a, b = z[..., 0::2], z[..., 1::2]
        z = torch.stack((a * c - b * n, b * c + a * n), -1).flatten(-2)
    else:
        a, b = z[..., :rot // 2], z[..., rot // 2:]
        z = torch.cat((a * c - b * n, b * c + a * n), -1)
    return torch.cat((z, rest), -1)


def _visible(p, j, window, sinks):
    return (j <= p) & ((j > p - window) | (j < sinks))


def _weights_plain(sc, seen):
    """Unnormalised weights of scores in 32 bits (overwritten) and their sums; rows that see nothing have 0 and 1."""
    sc = sc.masked_fill_(~seen, -math.inf)
    m = sc.amax(-1, keepdim=True)
    e = sc.sub_(torch.where(m.isinf(), torch.zeros_like(m), m)).exp_()
    n = e.sum(-1, keepdim=True)
    return e, torch.where(n > 0, n, torch.ones_like(n))


def _diff_plain(q, k, v, lam, weight, seen, scale):
    """q [B,2H,T,d], k, v [B,2Hk,J,d] in 32 bits, seen [B,1,T,J] -> [B,2H,T,d] in 32 bits."""
    B, H2, T, d = q.shape
    Hk, G = k.shape[1] // 2, H2 // k.shape[1]
    value = v.view(B, Hk, 2, -1, d).transpose(2, 3).reshape(B, Hk, -1, 2 * d)
    out = None
    for m in range(2):
        qm = q.view(B, Hk, G, 2, T, d)[:, :, :, m].reshape(B, Hk, G * T, d)
        sc = torch.matmul(qm * scale, k.view(B, Hk, 2, -1, d)[:, :, m].transpose(-1, -2)).view(B, Hk * G, T, -1)
        e, n = _weights_plain(sc, seen)
        o = torch.matmul(e.view(B, Hk, G * T, -1), value).view(B, Hk * G, T, 2 * d) / n
        out = o if m == 0 else out - lam[:, None, None] * o
    if weight is not None:
        out = out * torch.rsqrt(out.square().mean(-1, keepdim=True) + EPS) * weight
    return out.view(B, Hk * G, T, 2, d).transpose(2, 3).reshape(B, H2, T, d)


def run(s):
    case = s["case"]
    op, d, scale = case["op"], case["d"], case["d"] ** -0.5
    if op == "axes":
        if own:
            import gated_delta_rule_fwd_gb300 as lr
            cache = dict(v=s["v"], k_cache=s["k_cache"], v_cache=s["v_cache"], table=s["table"]) if case["append"] else {}
            lr.lr_qk_norm_rope_axes(s["q"], s["k"], s["positions"], s["axis"], s["places"], inv_freq=s["inv_freq"],
                                    interleaved=case["interleaved"], q_weight=s["qw"], k_weight=s["kw"], eps=EPS,
                                    q_out=s["q_out"], k_out=s["k_out"], **cache)
        else:
            kept = (s["places"] >= 0)[:, None, :, None]
            for x, w, y in ((s["q"], s["qw"], s["q_out"]), (s["k"], s["kw"], s["k_out"])):
                z = _axes_plain(x, w, s)
                y.copy_(torch.where(kept, z.to(y.dtype), y))
            if case["append"]:
                b, t = torch.nonzero(s["places"] >= 0, as_tuple=True)
                p = s["places"].long()[b, t]
                pages = s["table"].long()[b, p // case["page"]]
                s["k_cache"][pages, :, p % case["page"]] = s["k_out"][b, :, t]
                s["v_cache"][pages, :, p % case["page"]] = s["v"][b, :, t]
        out = dict(q=s["q_out"], k=s["k_out"])
        if case["append"]:
            out.update(k_cache=s["k_cache"], v_cache=s["v_cache"])
        return out
    if op == "diff":
        if own:
            import gated_delta_rule_fwd_gb300 as lr
            return lr.lr_fwd_diff(s["q"], s["k"], s["v"], s["lam"], window=case["window"], sinks=case["sinks"],
                                  q_len=s["q_len"], k_len=s["k_len"], scale=scale, norm=case["norm"],
                                  norm_weight=s["weight"], eps=EPS, o=s["o"])
        B, Tq, Tk = (case[n] for n in ("B", "Tq", "Tk"))
        dev = s["q"].device
        i, j = torch.arange(Tq, device=dev), torch.arange(Tk, device=dev)
        ql = torch.full((B,), Tq, device=dev) if s["q_len"] is None else s["q_len"].long()
        kl = torch.full((B,), Tk, device=dev) if s["k_len"] is None else s["k_len"].long()
        p = ((kl - ql)[:, None] + i)[:, :, None]
        live = (i[:, None] < ql[:, None, None])
        seen = _visible(p, j, case["window"], case["sinks"]) & (j < kl[:, None, None]) & live
        o = _diff_plain(s["q"].float(), s["k"].float(), s["v"].float(), s["lam"], s["weight"], seen[:, None], scale)
        s["o"].copy_(torch.where(live[:, None], o, s["o"].float()))
        return s["o"]
    N, Hk, page = case["N"], case["Hk"], case["page"]
    table, lens = s["table"].long(), s["lens"].long()
    most = table.shape[1] * page
    if op == "diff_step":
        if own:
            import gated_delta_rule_fwd_gb300 as lr
            return lr.lr_step_paged_diff(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"], s["lam"],
                                         max_len=case["len_hi"], window=case["window"], sinks=case["sinks"],
                                         scale=scale, norm=case["norm"], norm_weight=s["weight"], eps=EPS)
        k, v = (c[table].transpose(1, 2).reshape(N, 2 * Hk, most, d).float() for c in (s["k_cache"], s["v_cache"]))
        j = torch.arange(most, device=k.device)
        seen = _visible(lens[:, None] - 1, j, case["window"], case["sinks"])[:, None, None]
        o = _diff_plain(s["q"].float()[:, :, None], k, v, s["lam"], s["weight"], seen, scale)
        return o[:, :, 0].to(s["q"].dtype)
    if own:
        import gated_delta_rule_fwd_gb300 as lr
        return lr.lr_step_paged_prefix(s["q"], s["k_cache"], s["v_cache"], s["prefix"], case["P"], s["table"],
                                       s["lens"], max_len=case["len_hi"], window=case["window"],
                                       sinks=case["sinks"], scale=scale)
    Hq, P = case["Hq"], case["P"]
    q = s["q"].float().view(N, Hk, Hq // Hk, d) * scale
    # the prefix once for all sequences, then every sequence's own keys
    pk, pv = (c[s["prefix"].long()].transpose(0, 1).reshape(Hk, -1, d)[:, :P].float() for c in (s["k_cache"], s["v_cache"]))
    shared = torch.matmul(q.transpose(0, 1).reshape(Hk, -1, d), pk.transpose(-1, -2)).view(Hk, N, -1, P).transpose(0, 1)
    k, v = (c[table].transpose(1, 2).reshape(N, Hk, most, d).float() for c in (s["k_cache"], s["v_cache"]))
    sc = torch.cat((shared, torch.matmul(q, k.transpose(-1, -2))), -1)
    j = torch.arange(P + most, device=q.device)
    seen = _visible(P + lens[:, None] - 1, j, case["window"], case["sinks"])[:, None, None]
    e, n = _weights_plain(sc, seen)
    o = torch.matmul(e[..., :P].transpose(0, 1).reshape(Hk, -1, P), pv).view(Hk, N, -1, d).transpose(0, 1)
    o = (o + torch.matmul(e[..., P:], v)) / n
    return o.reshape(N, Hq, d).to(s["q"].dtype)


# -------------------------------------------------------------------- work

def _seen_counts(p, window, sinks):
    """How many keys positions p (>= 0) see: the window's, and the sinks before it."""
    p = np.asarray(p, np.int64)
    lo = np.maximum(p - window + 1, 0)
    return p - lo + 1 + np.minimum(np.minimum(lo, sinks), p + 1)


def work(case):
    es = 4 if case["dtype"] == "f32" else 2
    d, Hk, op = case["d"], case["Hk"], case["op"]
    if op == "axes":
        Hq = case["Hq"]
        rows = case["B"] * case["T"] * (0.5 if case["ragged"] else 1.0)
        vals = rows * (Hq + Hk) * d
        moved = 2 * vals + (3 * rows * Hk * d if case["append"] else 0)
        return {"bytes": moved * es + 4 * (case["axes"] + 1) * rows, "flops": 10 * vals}
    if op == "diff":
        B, Tq, Tk, H = case["B"], case["Tq"], case["Tk"], case["H"]
        pairs = float(_seen_counts(np.arange(Tk - Tq, Tk), case["window"], case["sinks"]).sum())
        part = (1 + (B - 1) * 0.5) if case["ragged"] else B
        reads = min(Tk, Tq + min(case["window"], Tk) + case["sinks"])
        return {"bytes": part * es * d * (4 * H * Tq + 4 * Hk * reads), "flops": 12 * d * H * pairs * part}
    N, W, S = case["N"], case["window"], case["sinks"]
    lens = np.linspace(case["len_lo"], case["len_hi"], 64)
    if op == "diff_step":
        seen = float(np.mean(_seen_counts(lens - 1, W, S))) * N
        return {"bytes": es * d * (4 * Hk * seen + 4 * case["H"] * N), "flops": 12 * d * case["H"] * seen}
    P, Hq = case["P"], case["Hq"]
    seen = float(np.mean(_seen_counts(P + lens - 1, W, S))) * N
    own_keys = float(np.mean(np.minimum(lens, W))) * N
    # of the prefix what any sequence sees
    shared = min(P, max(0, W - case["len_lo"]) + min(S, P))
    return {"bytes": es * d * (2 * Hk * (shared + own_keys) + 2 * Hq * N), "flops": 4 * d * Hq * seen}


# ------------------------------------------- the definition, in 64 bits

def _seen_rows(L, W, S, dev):
    """The keys that the last of L tokens sees."""
    lo = max(min(S, L), L - W)
    return torch.cat((torch.arange(min(S, lo), device=dev), torch.arange(lo, L, device=dev)))


def _normed64(o, weight):
    """o [..., 2d]: the root-mean-square norm, where there is one."""
    if weight is None:
        return o
    return o / ((o * o).sum(-1, keepdim=True) / o.shape[-1] + EPS).sqrt() * weight.double()


def exact(case, seed):
    s = prepare(case, seed)
    op, d, scale = case["op"], case["d"], case["d"] ** -0.5
    dev = s["q"].device
    if op == "axes":
        out = {}
        place, h = s["places"].long(), case["rot"] // 2
        kept = place >= 0
        th = torch.stack([s["positions"][a].double() * f for a, f in zip(s["axis"].tolist(), s["inv_freq"])], -1)
        turn = torch.complex(th.cos(), th.sin())[:, None]
        for n, w in (("q", s["qw"]), ("k", s["kw"])):
            x = s[n].double()
            x = x / (x.pow(2).sum(-1, keepdim=True) / d + EPS).sqrt() * w.double()
            # one complex number a pair, turned by e^{i p f}
            z = x[..., :2 * h]
            z = z.reshape(*z.shape[:-1], h, 2) if case["interleaved"] else z.reshape(*z.shape[:-1], 2, h).transpose(-1, -2)
            z = torch.view_as_real(torch.view_as_complex(z.contiguous()) * turn)
            z = z if case["interleaved"] else z.transpose(-1, -2)
            x = torch.cat((z.reshape(*x.shape[:-1], 2 * h), x[..., 2 * h:]), -1)
            out[n] = torch.where(kept[:, None, :, None], x, torch.zeros_like(x))
        if case["append"]:
            page, (total, Hk) = case["page"], s["k_cache"].shape[:2]
            slot = torch.gather(s["table"].long(), 1, place.clamp(min=0) // page) * page + place.clamp(min=0) % page
            for n, src in (("k_cache", out["k"]), ("v_cache", s["v"].double())):
                flat = torch.zeros(total * page, Hk, d, dtype=torch.float64, device=dev)
                flat[slot[kept]] = src.transpose(1, 2)[kept]
                out[n] = flat.view(total, page, Hk, d).transpose(1, 2)
        return out
    W, S, Hk = case["window"], case["sinks"], case["Hk"]
    if op in ("prefix", "diff_step"):
        N, page = case["N"], case["page"]
        if N * Hk > 4096 or work(case)["flops"] > 1e12:
            return None
        o = torch.zeros(s["q"].shape, dtype=torch.float64, device=dev)
        q, table = s["q"].double(), s["table"].long()
        for n, L in enumerate(s["lens"].tolist()):
            if op == "prefix":
                P = case["P"]
                j = _seen_rows(P + L, W, S, dev)
                i = (j - P).clamp(min=0)
                where = torch.where(j < P, s["prefix"].long()[j.clamp(max=P - 1) // page], table[n, i // page])
                at = torch.where(j < P, j % page, i % page)
            else:
                j = _seen_rows(L, W, S, dev)
                where, at = table[n, j // page], j % page
            k, v = (c[where, :, at].double().transpose(0, 1) for c in (s["k_cache"], s["v_cache"]))
            if op == "prefix":
                qn = q[n].view(Hk, -1, d)
                o[n] = (torch.softmax(qn @ k.transpose(1, 2) * scale, -1) @ v).reshape(-1, d)
            else:
                qn = q[n].view(Hk, -1, 2, d).permute(2, 0, 1, 3)
                value = torch.cat((v[0::2], v[1::2]), -1)
                a = [torch.softmax(qn[m] @ k[m::2].transpose(1, 2) * scale, -1) @ value for m in range(2)]
                y = (a[0] - s["lam"].double().view(Hk, -1, 1) * a[1]).reshape(-1, 2 * d)
                o[n] = _normed64(y, s["weight"]).reshape(-1, d)
        return o
    B, H, Tq, Tk = case["B"], case["H"], case["Tq"], case["Tk"]
    G = H // Hk
    if work(case)["flops"] > 2e12:
        return None
    o = torch.zeros(B, 2 * H, Tq, d, dtype=torch.float64, device=dev)
    step = 512
    for b in range(B):
        ql = Tq if s["q_len"] is None else int(s["q_len"][b])
        kl = Tk if s["k_len"] is None else int(s["k_len"][b])
        for i0 in range(0, ql, step):
            i1 = min(ql, i0 + step)
            p = torch.arange(kl - ql + i0, kl - ql + i1, device=dev)[:, None]
            first = max(min(S, kl), int(p[0]) - W + 1)
            j = torch.cat((torch.arange(min(S, first), device=dev), torch.arange(first, max(first, int(p[-1]) + 1), device=dev)))
            hidden = (j > p) | ((j <= p - W) & (j >= S))
            for h in range(H):
                value = torch.cat((s["v"][b, 2 * (h // G), j], s["v"][b, 2 * (h // G) + 1, j]), -1).double()
                y = 0
                for m in range(2):
                    sc = (s["q"][b, 2 * h + m, i0:i1].double() @ s["k"][b, 2 * (h // G) + m, j].double().T) * scale
                    part = torch.softmax(sc.masked_fill(hidden, -math.inf), -1) @ value
                    y = part if m == 0 else y - s["lam"][h].double() * part
                y = _normed64(y, s["weight"])
                o[b, 2 * h, i0:i1], o[b, 2 * h + 1, i0:i1] = y[:, :d], y[:, d:]
    return o
