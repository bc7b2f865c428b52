"""Cases that measure the attention operators beside the linear-attention
mixers: the norm and rotation of queries and keys (with the write into a paged
cache), attention with a sliding window and sink tokens over whole sequences,
and its step for single tokens over the paged cache.

``own`` false: plain torch; true: this repository's entry points.
"""
import math

import numpy as np
import torch

own = False

NO_WINDOW = 1 << 30


def _dev():
    return torch.device("cuda" if torch.cuda.is_available() else "cpu")


def _dt(case):
    return torch.float32 if case["dtype"] == "f32" else torch.bfloat16


def listed():
    return [
        # one decode step of a 64-sequence batch: q, k, v of one token each, k and v into the pages
        dict(name="norm_rope_step", op="norm_rope", dtype="bf16", B=64, T=1, Hq=32, Hk=8, d=128, rot=128,
             interleaved=False, far=30000, page=64, append=True, ragged=False),
        # the prompts of two sequences, at the sizes of the gated-delta prefill workload
        dict(name="norm_rope_prefill", op="norm_rope", dtype="bf16", B=2, T=16384, Hq=16, Hk=4, d=128, rot=128,
             interleaved=False, far=0, page=64, append=False, ragged=False),
        # an odd, padded fp32 batch, interleaved pairs, half of the channels rotated, far positions, appended
        dict(name="norm_rope_odd", op="norm_rope", dtype="f32", B=3, T=777, Hq=6, Hk=2, d=64, rot=32,
             interleaved=True, far=1000000, page=16, append=True, ragged=True),
        # short padded prompts: latency
        dict(name="window_short", op="window", dtype="bf16", B=4, Hq=8, Hk=2, Tq=173, Tk=173, d=64, window=64,
             sinks=4, ragged=True),
        # a middle-sized batch (the retention workload's), a head each for queries and keys
        dict(name="window_mid", op="window", dtype="bf16", B=4, Hq=8, Hk=8, Tq=2048, Tk=2048, d=128, window=512,
             sinks=4, ragged=False),
        # one long prompt with shared key heads
        dict(name="window_long", op="window", dtype="bf16", B=1, Hq=16, Hk=4, Tq=16384, Tk=16384, d=128, window=1024,
             sinks=4, ragged=False),
        # no limit but causality: the layer without a window
        dict(name="window_causal", op="window", dtype="bf16", B=2, Hq=16, Hk=16, Tq=4096, Tk=4096, d=128,
             window=NO_WINDOW, sinks=0, ragged=False),
        # a later piece of padded prompts in fp32, odd sizes
        dict(name="window_f32_piece", op="window", dtype="f32", B=2, Hq=8, Hk=2, Tq=700, Tk=1501, d=64, window=300,
             sinks=3, ragged=True),
        # one sequence being answered: latency
        dict(name="step_one", op="step", dtype="bf16", N=1, Hq=32, Hk=8, d=128, len_lo=1200, len_hi=1200, page=64,
             window=NO_WINDOW, sinks=0),
        # a serving batch of very different lengths
        dict(name="step_batch", op="step", dtype="bf16", N=128, Hq=32, Hk=8, d=128, len_lo=500, len_hi=8192, page=64,
             window=NO_WINDOW, sinks=0),
        # two sequences with a long cache: the work is split over its length
        dict(name="step_long", op="step", dtype="bf16", N=2, Hq=16, Hk=4, d=128, len_lo=131000, len_hi=131072, page=128,
             window=NO_WINDOW, sinks=0),
        # fp32, window and sinks, odd lengths, some shorter than the window
        dict(name="step_f32_window", op="step", dtype="f32", N=33, Hq=8, Hk=8, d=64, len_lo=1, len_hi=5000, page=16,
             window=1024, sinks=4),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm_rope", "window", "step"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    d = rng.choice([32, 64, 128])
    Hk = rng.choice([1, 2, 3, 4, 8])
    group = rng.choice([1, 2, 3, 4, 8])
    Hq = Hk * group
    if op == "norm_rope":
        B = _log(rng, 1, 64)
        T = _log(rng, 1, max(1, min(16384, (2 * 16384 * 20 * 128) // (B * (Hq + Hk) * d))))
        rot = rng.choice([d, d, d // 2, 0])
        append = rng.random() < 0.5
        return dict(op=op, dtype=dtype, B=B, T=T, Hq=Hq, Hk=Hk, d=d, rot=rot, interleaved=rng.random() < 0.5,
                    far=rng.choice([0, 5000, 1000000]), page=rng.choice([16, 32, 64, 128]), append=append,
                    ragged=append and rng.random() < 0.5)
    if op == "window":
        B = _log(rng, 1, 8)
        Tk = _log(rng, 1, 8192 if dtype == "bf16" else 2048)
        while B > 1 and B * Hq * Tk * Tk > 16 * 8192 * 8192:
            B -= 1
        while Hk > 1 and B * Hq * Tk * Tk > 16 * 8192 * 8192:
            Hk -= 1
            Hq = Hk * group
        Tq = Tk if rng.random() < 0.6 else _log(rng, 1, Tk)
        window = NO_WINDOW if rng.random() < 0.3 else _log(rng, 1, 4096)
        return dict(op=op, dtype=dtype, B=B, Hq=Hq, Hk=Hk, Tq=Tq, Tk=Tk, d=d, window=window,
                    sinks=rng.choice([0, 1, 4, 5, 64]), ragged=rng.random() < 0.5)
    N = _log(rng, 1, 128)
    hi = _log(rng, 1, max(1, min(131072, (128 * 8192 * 8 * 128) // (N * Hk * d * (2 if dtype == "f32" else 1)))))
    return dict(op=op, dtype=dtype, N=N, Hq=Hq, Hk=Hk, d=d, len_lo=max(1, hi // rng.choice([1, 2, 16])), len_hi=hi,
                page=rng.choice([16, 32, 64, 128]), window=NO_WINDOW if rng.random() < 0.5 else _log(rng, 1, 4096),
                sinks=rng.choice([0, 1, 4, 5, 64]))


# ------------------------------------------------------------------ inputs

def _lengths(case, seed):
    """The lengths of a step's sequences: from the case alone in count and range, drawn from the seed; the longest is there."""
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


def prepare(case, seed):
    dev, dt = _dev(), _dt(case)
    g = torch.Generator(dev)
    g.manual_seed(int(seed) * 7919 + 17)
    r = np.random.RandomState((int(seed) * 31 + 5) % (1 << 31))

    def normal(*shape, std=1.0, dtype=dt):
        return (torch.randn(*shape, generator=g, device=dev, dtype=torch.float32) * std).to(dtype)

    s = dict(case=case)
    d = case["d"]
    if case["op"] == "norm_rope":
        B, T, Hq, Hk = case["B"], case["T"], case["Hq"], case["Hk"]
        # one projection's output, tokens first: q, k and v are views of it
        x = normal(B, T, Hq + 2 * Hk, d)
        s["q"], s["k"], s["v"] = (x[:, :, a:b].transpose(1, 2) for a, b in ((0, Hq), (Hq, Hq + Hk), (Hq + Hk, Hq + 2 * Hk)))
        s["qw"] = 1 + normal(d, std=0.1, dtype=torch.float32)
        s["kw"] = 1 + normal(d, std=0.1, dtype=torch.float32)
        half = case["rot"] // 2
        s["inv_freq"] = None
        if half:
            s["inv_freq"] = 10000.0 ** (-torch.arange(half, dtype=torch.float64, device=dev) / half)
        first = r.randint(case["far"] // 2, case["far"] + 1, (B, 1))
        pos = first + np.arange(T)
        if case["ragged"]:  # rows behind a prompt's end are padding
            pos[np.arange(T) >= r.randint(0, T + 1, (B, 1))] = -1
        s["q_out"] = torch.zeros(B, Hq, T, d, dtype=dt, device=dev)
        s["k_out"] = torch.zeros(B, Hk, T, d, dtype=dt, device=dev)
        s["positions"] = torch.from_numpy(pos.astype(np.int32)).to(dev)
        if case["append"]:
            page = case["page"]
            # pages of positions before this piece are not in the pool (evicted): they share page 0
            held = [(int(f) // page, (int(f) + T - 1) // page) for f in first[:, 0]]
            most = max(b for _, b in held) + 1
            table = np.zeros((B, most), np.int32)
            total = sum(b - a + 1 for a, b in held) + 1
            order = 1 + r.permutation(total - 1).astype(np.int32)
            at = 0
            for n, (a, b) in enumerate(held):
                table[n, a:b + 1] = order[at:at + b - a + 1]
                at += b - a + 1
            s["table"] = torch.from_numpy(table).to(dev)
            s["k_cache"] = torch.zeros(total, Hk, page, d, dtype=dt, device=dev)
            s["v_cache"] = torch.zeros(total, Hk, page, d, dtype=dt, device=dev)
    elif case["op"] == "window":
        B, Hq, Hk, Tq, Tk = (case[n] for n in ("B", "Hq", "Hk", "Tq", "Tk"))
        # normed queries and keys, in the library's layout, and values as the projection leaves them
        s["q"], s["k"] = normal(B, Hq, Tq, d), normal(B, Hk, Tk, d)
        s["v"] = normal(B, Tk, Hk, d).transpose(1, 2)
        s["q_len"] = s["k_len"] = None
        if case["ragged"]:
            ql = r.randint(0 if B > 1 else 1, Tq + 1, B)
            ql[0] = Tq
            kl = np.minimum(ql + r.randint(0, Tk - Tq + 1, B), Tk)
            s["q_len"], s["k_len"] = (torch.from_numpy(a.astype(np.int32)).to(dev) for a in (ql, kl))
        s["o"] = torch.zeros(B, Hq, Tq, d, dtype=dt, device=dev)
    else:
        lens = _lengths(case, int(seed))
        table, total = _pages(r, lens, case["page"])
        s["q"] = normal(case["N"], case["Hq"], d)
        s["k_cache"] = normal(total, case["Hk"], case["page"], d)
        s["v_cache"] = normal(total, case["Hk"], case["page"], d)
        s["table"], s["lens"] = torch.from_numpy(table).to(dev), torch.from_numpy(lens).to(dev)
    return s


# ------------------------------------------------------------- the operators

def _norm_rope_plain(x, w, inv_freq, positions, interleaved):
    """x [B,H,T,d] -> 32 bits; angles in 64."""
    y = x.float()
    y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6) * w
    if inv_freq is None:
        return y
    rot = 2 * inv_freq.numel()
    th = positions.double()[:, None, :, None] * inv_freq
    c, s = torch.cos(th).float(), torch.sin(th).float()
    z, rest = y[..., :rot], y[..., rot:]
    if interleaved:
        a, b = z[..., 0::2], z[..., 1::2]
        z = torch.stack((a * c - b * s, b * c + a * s), -1).flatten(-2)
    else:
        a, b = z[..., :rot // 2], z[..., rot // 2:]
        z = torch.cat((a * c - b * s, b * c + a * s), -1)
    return torch.cat((z, rest), -1)


def _visible(p, j, window, sinks):
    return (j <= p) & ((j > p - window) | (j < sinks))


def _attend_plain(q, k, v, seen, scale):
    """q [B,Hk,G,T,d], k, v [B,Hk,J,d] in 32 bits, seen [B,1,1,T,J]: rows that see nothing are 0."""
    B, Hk, G, T, d = q.shape
    sc = torch.matmul((q * scale).flatten(2, 3), k.transpose(-1, -2)).view(B, Hk, G, T, -1)
    sc = sc.masked_fill_(~seen, -math.inf)
    m = sc.amax(-1, keepdim=True)
    e = sc.sub_(torch.where(m.isinf(), torch.zeros_like(m), m)).exp_()
    l = e.sum(-1, keepdim=True)
    return torch.matmul(e.flatten(2, 3), v).view(B, Hk, G, T, d) / torch.where(l > 0, l, torch.ones_like(l))


def run(s):
    case = s["case"]
    d, scale = case["d"], case["d"] ** -0.5
    if case["op"] == "norm_rope":
        if own:
            import gated_delta_rule_fwd_gb300 as lr
            cache = dict(v=s["v"], k_cache=s["k_cache"], v_cache=s["v_cache"], table=s["table"]) if case["append"] else {}
            lr.lr_qk_norm_rope(s["q"], s["k"], s["positions"], inv_freq=s["inv_freq"],
                               interleaved=case["interleaved"], q_weight=s["qw"], k_weight=s["kw"], eps=1e-6,
                               q_out=s["q_out"], k_out=s["k_out"], **cache)
        else:
            kept = (s["positions"] >= 0)[:, None, :, None]
            for x, w, y in ((s["q"], s["qw"], s["q_out"]), (s["k"], s["kw"], s["k_out"])):
                z = _norm_rope_plain(x, w, s["inv_freq"], s["positions"], case["interleaved"])
                y.copy_(torch.where(kept, z.to(y.dtype), y))
            if case["append"]:
                pos = s["positions"].long()
                b, t = torch.nonzero(pos >= 0, as_tuple=True)
                p = pos[b, t]
                pages = s["table"].long()[b, p // case["page"]]
                s["k_cache"][pages, :, p % case["page"]] = s["k_out"][b, :, t]
                s["v_cache"][pages, :, p % case["page"]] = s["v"][b, :, t]
        out = dict(q=s["q_out"], k=s["k_out"])
        if case["append"]:
            out.update(k_cache=s["k_cache"], v_cache=s["v_cache"])
        return out
    if case["op"] == "window":
        if own:
            import gated_delta_rule_fwd_gb300 as lr
            return lr.lr_fwd_window(s["q"], s["k"], s["v"], window=case["window"], sinks=case["sinks"],
                                    q_len=s["q_len"], k_len=s["k_len"], scale=scale, o=s["o"])
        B, Hq, Hk, Tq, Tk = (case[n] for n in ("B", "Hq", "Hk", "Tq", "Tk"))
        dev = s["q"].device
        i, j = torch.arange(Tq, device=dev), torch.arange(Tk, device=dev)
        ql = torch.full((B,), Tq, device=dev) if s["q_len"] is None else s["q_len"].long()
        kl = torch.full((B,), Tk, device=dev) if s["k_len"] is None else s["k_len"].long()
        p = ((kl - ql)[:, None] + i)[:, :, None]
        seen = _visible(p, j, case["window"], case["sinks"]) & (j < kl[:, None, None]) & (i[:, None] < ql[:, None, None])
        o = _attend_plain(s["q"].float().view(B, Hk, Hq // Hk, Tq, d), s["k"].float(), s["v"].float(),
                          seen[:, None, None], scale).view(B, Hq, Tq, d)
        s["o"].copy_(o)
        return s["o"]
    if own:
        import gated_delta_rule_fwd_gb300 as lr
        return lr.lr_step_paged(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"], max_len=case["len_hi"],
                                window=case["window"], sinks=case["sinks"], scale=scale)
    N, Hq, Hk, page = (case[n] for n in ("N", "Hq", "Hk", "page"))
    table, lens = s["table"].long(), s["lens"].long()
    most = table.shape[1]
    k, v = (c[table].transpose(1, 2).reshape(N, Hk, most * page, d).float() for c in (s["k_cache"], s["v_cache"]))
    j = torch.arange(most * page, device=k.device)
    seen = _visible(lens[:, None] - 1, j, case["window"], case["sinks"])[:, None, None, None]
    o = _attend_plain(s["q"].float().view(N, Hk, Hq // Hk, 1, d), k, v, seen, scale)
    return o.view(N, Hq, d).to(s["q"].dtype)


# -------------------------------------------------------------------- work

def _seen_counts(p, window, sinks):
    """How many keys positions p (>= 0) see: the window's, and the sinks before it."""
    p = np.asarray(p, np.int64)
    lo = np.maximum(p - window + 1, 0)
    return p - lo + 1 + np.minimum(np.minimum(lo, sinks), p + 1)


def work(case):
    es = 4 if case["dtype"] == "f32" else 2
    d, Hq, Hk = case["d"], case["Hq"], case["Hk"]
    if case["op"] == "norm_rope":
        rows = case["B"] * case["T"] * (0.5 if case["ragged"] else 1.0)
        vals = rows * (Hq + Hk) * d
        moved = 2 * vals + (3 * rows * Hk * d if case["append"] else 0)
        return {"bytes": moved * es, "flops": 10 * vals}
    if case["op"] == "window":
        B, Tq, Tk = case["B"], case["Tq"], case["Tk"]
        pairs = float(_seen_counts(np.arange(Tk - Tq, Tk), case["window"], case["sinks"]).sum())
        part = (1 + (B - 1) * 0.5) if case["ragged"] else B
        reads = min(Tk, Tq + min(case["window"], Tk) + case["sinks"])
        return {"bytes": part * es * d * (2 * Hq * Tq + 2 * Hk * reads), "flops": 4 * d * Hq * pairs * part}
    mean = (case["len_lo"] + case["len_hi"]) / 2
    seen = min(mean, min(case["window"], mean) + case["sinks"]) * case["N"]
    return {"bytes": es * d * (2 * Hk * seen + 2 * Hq * case["N"]), "flops": 4 * d * Hq * seen}


# ------------------------------------------- the definition, in 64 bits

def _rows64(q, k, v, scale):
    """Attention of rows q [G,d] or [G,T,d] with a list of keys they all see."""
    a = torch.softmax((q @ k.T) * scale, -1)
    return a @ v


def exact(case, seed):
    s = prepare(case, seed)
    d, scale = case["d"], case["d"] ** -0.5
    if case["op"] == "norm_rope":
        out = {}
        pos = s["positions"]
        kept = pos >= 0
        for n, w in (("q", s["qw"]), ("k", s["kw"])):
            x = s[n].double()
            x = x / (x.pow(2).sum(-1, keepdim=True) / d + 1e-6).sqrt() * w.double()
            h = case["rot"] // 2
            if h:
                # one complex number a pair, turned by e^{i p f}
                z = x[..., :2 * h]
                z = z.reshape(*z.shape[:-1], h, 2) if case["interleaved"] else z.reshape(*z.shape[:-1], 2, h).transpose(-1, -2)
                th = pos.double()[:, None, :, None] * s["inv_freq"]
                turn = torch.complex(th.cos(), th.sin())
                z = torch.view_as_real(torch.view_as_complex(z.contiguous()) * turn)
                z = z if case["interleaved"] else z.transpose(-1, -2)
                x = torch.cat((z.reshape(*x.shape[:-1], 2 * h), x[..., 2 * h:]), -1)
            out[n] = torch.where(kept[:, None, :, None], x, torch.zeros_like(x))
        if case["append"]:
            page, (total, Hk) = case["page"], s["k_cache"].shape[:2]
            slot = torch.gather(s["table"].long(), 1, pos.long().clamp(min=0) // page) * page + pos.long().clamp(min=0) % page
            for n, src in (("k_cache", out["k"]), ("v_cache", s["v"].double())):
                flat = torch.zeros(total * page, Hk, d, dtype=torch.float64, device=src.device)
                flat[slot[kept]] = src.transpose(1, 2)[kept]
                out[n] = flat.view(total, page, Hk, d).transpose(1, 2)
        return out
    Hq, Hk, W, S = case["Hq"], case["Hk"], case["window"], case["sinks"]
    G = Hq // Hk
    if case["op"] == "step":
        if case["N"] * Hk > 4096:
            return None
        o = torch.zeros(case["N"], Hq, d, dtype=torch.float64, device=s["q"].device)
        table = s["table"].long()
        for n, L in enumerate(s["lens"].tolist()):
            lo = max(min(S, L), L - W)
            rows = torch.cat((torch.arange(min(S, lo), device=o.device), torch.arange(lo, L, device=o.device)))
            where = (table[n, rows // case["page"]], slice(None), rows % case["page"])
            k, v = s["k_cache"][where].double(), s["v_cache"][where].double()
            for h in range(Hk):
                o[n, h * G:(h + 1) * G] = _rows64(s["q"][n, h * G:(h + 1) * G].double(), k[:, h], v[:, h], scale)
        return o
    B, Tq, Tk = case["B"], case["Tq"], case["Tk"]
    if work(case)["flops"] > 1.5e12:
        return None
    o = torch.zeros(B, Hq, Tq, d, dtype=torch.float64, device=s["q"].device)
    step = 512
    for b in range(B):
        ql = Tq if s["q_len"] is None else int(s["q_len"][b])
        kl = Tk if s["k_len"] is None else int(s["k_len"][b])
        for i0 in range(0, ql, step):
            i1 = min(ql, i0 + step)
            p = torch.arange(kl - ql + i0, kl - ql + i1, device=o.device)[:, None]
            first = max(min(S, kl), int(p[0]) - W + 1)
            j = torch.cat((torch.arange(min(S, first), device=o.device), torch.arange(first, max(first, int(p[-1]) + 1), device=o.device)))
            hidden = (j > p) | ((j <= p - W) & (j >= S))
            for h in range(Hk):
                k, v = s["k"][b, h, j].double(), s["v"][b, h, j].double()
                sc = (s["q"][b, h * G:(h + 1) * G, i0:i1].double() @ k.T) * scale
                o[b, h * G:(h + 1) * G, i0:i1] = torch.softmax(sc.masked_fill(hidden, -math.inf), -1) @ v
    return o
