"""lr_step_paged_prefix against its fp64 definition (oracle/attention.py),
element by element within ``attention_bound``, and against lr_step_paged over
the same tokens.
"""
import numpy as np
import pytest
import torch

import gated_delta_rule_fwd_gb300 as lr
from oracle import attention as oa

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
BITS = {F32: 24, BF16: 8}          # half a step of the type, 2^-bits relative
NW = lr.NO_WINDOW
LR_OK, LR_ERR_INDEX = 0, 13
types = pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
CUTS = [64, 700, 40000]   # bounds on the length: one chunk, a cluster's few, many joined by a kernel


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from gated_delta_rule_fwd_gb300.build import build
    build()
    lr.device_status()
    yield torch.device("cuda:0")
    assert lr.device_status() == LR_OK


def rnd(seed, *shape, dtype=F32, std=1.0):
    g = torch.Generator("cpu").manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std).to(dtype)


def np64(t):
    return t.detach().cpu().double().numpy()


def within(got, want, bound):
    got = np64(got)
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), (f"{bad.sum()} of {bad.size} outside, first at {np.argwhere(bad)[0]}: "
                           f"{got[bad][0]} for {want[bad][0]} +- {bound[bad][0]}")


def paged(seed, lens, Hk, page, d, dtype, dev, extra=2):
    """Pools with the sequences' pages in no order and NaN everywhere else."""
    r = np.random.RandomState(seed)
    need = [max(0, -(-max(L, 0) // page)) for L in lens]
    total, most = sum(need) + extra, max(1, max(need)) + 1
    order = r.permutation(total)
    table = r.randint(0, total, (len(lens), most)).astype(np.int32)
    kc, vc = (torch.full((total, Hk, page, d), float("nan"), dtype=dtype) for _ in range(2))
    at = 0
    for n, L in enumerate(lens):
        for j in range(need[n]):
            pg = int(order[at])
            at += 1
            table[n, j] = pg
            rows = min(page, L - j * page)
            kc[pg, :, :rows] = rnd(seed + 31 * at, Hk, rows, d, dtype=dtype)
            vc[pg, :, :rows] = rnd(seed + 31 * at + 7, Hk, rows, d, dtype=dtype)
    return kc.to(dev), vc.to(dev), torch.from_numpy(table).to(dev)


def shared(seed, P, lens, Hk, page, d, dtype, dev):
    """Pools, the prefix's pages and the own tokens' table."""
    kc, vc, table = paged(seed, list(lens) + [P], Hk, page, d, dtype, dev)
    return kc, vc, table[-1, :-(-P // page)].contiguous(), table[:-1, :max(1, -(-max(max(lens), 1) // page))].contiguous()


def wider(table, max_len, page, dev):
    wide = torch.zeros(table.shape[0], -(-max_len // page), dtype=torch.int32, device=dev)
    most = min(wide.shape[1], table.shape[1])
    wide[:, :most] = table[:, :most]
    return wide


def check(dev, q, kc, vc, prefix, P, table, lens, window, sinks, scale=None, max_len=None, **kw):
    dtype, d = q.dtype, q.shape[-1]
    scale = d ** -0.5 if scale is None else scale
    o = torch.full(q.shape, 7.0, dtype=dtype, device=dev)
    ld = torch.tensor(lens, dtype=torch.int32, device=dev)
    args = dict(max_len=max_len, window=window, sinks=sinks, scale=scale, **kw)
    out = lr.lr_step_paged_prefix(q.to(dev), kc, vc, prefix, P, table, ld, o=o, **args)
    torch.cuda.synchronize()
    assert out is o
    ref, size, reach, written = oa.step_prefix(np64(q), np64(kc), np64(vc), prefix.cpu().numpy(), P, table.cpu().numpy(),
                                               lens, window, sinks, scale)
    bound = oa.attention_bound(ref, size, reach, P + max(max(lens), 1), d, BITS[dtype], 8 if dtype == BF16 else None)
    w = np.broadcast_to(written[:, None, None], ref.shape)
    within(out, np.where(w, ref, 7.0), np.where(w, bound, 0.0))
    made = lr.lr_step_paged_prefix(q.to(dev), kc, vc, prefix, P, table, ld, **args)
    assert torch.equal(made, torch.where(torch.from_numpy(w.copy()).to(dev), out, torch.zeros_like(out)))
    return out


LENS = [1, 0, 15, 16, 17, -1, 127, 128, 129, 300]


@types
@pytest.mark.parametrize("d,Hq,Hk", [(32, 4, 2), (64, 17, 1), (128, 6, 2), (128, 3, 3)])
@pytest.mark.parametrize("P", [0, 1, 15, 16, 127, 128, 129, 300, 1000])
@pytest.mark.parametrize("page,window,sinks", [(16, NW, 0), (64, 140, 5), (256, 400, 200)])
def test_prefix_parity(dev, dtype, d, Hq, Hk, P, page, window, sinks):
    """Prefixes that end inside tiles and pages, own lengths of zero, one and
    page edges, unused slots; windows that leave the prefix behind for some rows;
    sinks beyond a short prefix; NaN in every row of the pools that no one holds."""
    kc, vc, prefix, table = shared(P + d + Hq, P, LENS, Hk, page, d, dtype, dev)
    check(dev, rnd(30, len(LENS), Hq, d, dtype=dtype), kc, vc, prefix, P, table, LENS, window, sinks)


@types
@pytest.mark.parametrize("N,Hq,Hk", [(1, 1, 1), (1, 8, 1), (33, 4, 1), (64, 2, 1), (65, 2, 1), (129, 2, 2), (70, 16, 4),
                                     (300, 1, 1)])
@pytest.mark.parametrize("window,sinks", [(NW, 0), (350, 3)])
def test_prefix_numbers_of_rows(dev, dtype, N, Hq, Hk, window, sinks):
    """From one row to several blocks of them, the last one ragged."""
    d, P = 64, 400
    lens = [(7 * n) % 40 - (n % 11 == 3) * 50 for n in range(N)]
    kc, vc, prefix, table = shared(N, P, lens, Hk, 32, d, dtype, dev)
    check(dev, rnd(31, N, Hq, d, dtype=dtype), kc, vc, prefix, P, table, lens, window, sinks)


@types
@pytest.mark.parametrize("max_len,window,sinks", [(64, NW, 0), (700, NW, 0), (4097, NW, 0), (40000, NW, 0),
                                                  (20000, 300, 0), (20000, 300, 7), (20000, 4000, 2500)])
def test_prefix_cut_by_the_bound_on_the_length(dev, dtype, max_len, window, sinks):
    """Own tokens in one chunk, in a cluster's few, in many joined by a kernel;
    a prefix in many parts."""
    lens, P = [x for x in (1, 0, 64, -1, 63, 700, 4000) if x <= max_len], 2300
    kc, vc, prefix, table = shared(21, P, lens, 2, 64, 64, dtype, dev)
    check(dev, rnd(37, len(lens), 6, 64, dtype=dtype), kc, vc, prefix, P, wider(table, max_len, 64, dev), lens, window,
          sinks, max_len=max_len)


@types
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (33, 50), (250, 17), (290, 0), (310, 300), (NW, 4)])
@pytest.mark.parametrize("page", [16, 128])
def test_prefix_sees_each_key_once(dev, dtype, window, sinks, page):
    """Zero keys, values that mark the key."""
    d, lens, P = 128, [40, 1, 0], 270
    kc, vc, prefix, table = shared(3, P, lens, 1, page, d, dtype, dev)
    for pages, L in [(prefix, P)] + [(table[n], lens[n]) for n in range(3)]:
        for j in range(L):
            pg, mark = int(pages[j // page]), j + (0 if pages is prefix else P)
            kc[pg, 0, j % page] = 0
            vc[pg, 0, j % page] = 0
            vc[pg, 0, j % page, mark % d] = 1
    check(dev, rnd(31, 3, 2, d, dtype=dtype), kc, vc, prefix, P, table, lens, window, sinks, 1.0)


@types
@pytest.mark.parametrize("d", [32, 64, 128])
def test_prefix_is_the_step_over_the_same_tokens(dev, dtype, d):
    """A prefix of whole pages: lr_step_paged with its pages before each
    sequence's own gives the same, each within the bound of the definition."""
    page, P, lens = 64, 64 * 30, [5, 100, 64, 1]
    kc, vc, prefix, table = shared(41, P, lens, 2, page, d, dtype, dev)
    q = rnd(42, 4, 8, d, dtype=dtype)
    for window, sinks in ((NW, 0), (1000, 4)):
        a = check(dev, q, kc, vc, prefix, P, table, lens, window, sinks)
        whole = torch.cat((prefix.expand(4, -1), table), 1).contiguous()
        b = lr.lr_step_paged(q.to(dev), kc, vc, whole, torch.tensor(lens, dtype=torch.int32, device=dev) + P,
                             window=window, sinks=sinks)
        ref, size, reach, _ = oa.step_prefix(np64(q), np64(kc), np64(vc), prefix.cpu().numpy(), P, table.cpu().numpy(),
                                             lens, window, sinks, d ** -0.5)
        bound = oa.attention_bound(ref, size, reach, P + 100, d, BITS[dtype], 8 if dtype == BF16 else None)
        within(b, ref, bound)
        within(a, np64(b), 2 * bound)


@types
@pytest.mark.parametrize("max_len", CUTS)
@pytest.mark.parametrize("scale", [0.0, -0.4, 1e-3, 3.0])
def test_prefix_scales(dev, dtype, scale, max_len):
    lens, P = [64, 3, 0], 200
    kc, vc, prefix, table = shared(22, P, lens, 1, 16, 64, dtype, dev)
    check(dev, rnd(23, 3, 4, 64, dtype=dtype), kc, vc, prefix, P, wider(table, max_len, 16, dev), lens, NW, 0, scale,
          max_len=max_len)


@types
def test_prefix_masked_keys_may_hold_anything(dev, dtype):
    """Keys between the sinks and the windows are NaN and infinite, in the
    prefix and among the own tokens."""
    lens, d, page, P = [130, 9], 128, 32, 400
    kc, vc, prefix, table = shared(6, P, lens, 2, page, d, dtype, dev)
    q = rnd(33, 2, 8, d, dtype=dtype)
    want = check(dev, q, kc, vc, prefix, P, table, lens, 100, 5)
    for j in range(5, P + 9 - 100):
        kc[int(prefix[j // page]), :, j % page] = float("nan") if j % 2 else float("inf")
        vc[int(prefix[j // page]), :, j % page] = float("inf") if j % 3 else float("nan")
    for j in range(0, 30):
        vc[int(table[0, j // page]), :, j % page] = float("nan")
    got = lr.lr_step_paged_prefix(q.to(dev), kc, vc, prefix, P, table, torch.tensor(lens, dtype=torch.int32, device=dev),
                                  window=100, sinks=5)
    ref, size, reach, _ = oa.step_prefix(*(np64(t) for t in (q, kc, vc)), prefix.cpu().numpy(), P, table.cpu().numpy(),
                                         lens, 100, 5, d ** -0.5)
    bound = oa.attention_bound(ref, size, reach, 600, d, BITS[dtype], 8 if dtype == BF16 else None)
    within(got, ref, bound)
    within(want, ref, bound)


@types
@pytest.mark.parametrize("d,Hq,Hk", [(32, 2, 1), (64, 17, 1), (128, 6, 2)])
@pytest.mark.parametrize("max_len", CUTS)
def test_prefix_values_that_are_not_finite_or_overflow_a_sum(dev, max_len, d, Hq, Hk, dtype):
    """As for lr_step_paged: a channel with a seen infinity is that infinity (of
    a key whose weight underflows, too), with both signs or a NaN it is NaN, any
    other is as without them; values near the type's end average without overflow;
    a page outside the pool is left out."""
    page, inf, nan, lens, P = 16, float("inf"), float("nan"), [50, 61, 0, 33], 150
    kc, vc, prefix, table = shared(130, P, lens, Hk, page, d, dtype, dev)
    q = rnd(131, len(lens), Hq, d, dtype=dtype)
    place = lambda pages, j: (int(pages[j // page]), slice(None), j % page)
    q[0] = 1
    kc[place(prefix, 9)] = -1e4      # for sequence 0 a score of -1e4 sqrt(d): no weight
    # the prefix's third page is outside the pool
    broken = prefix.clone()
    broken[2] = -1
    left = [j for j in range(P) if j // page != 2]
    def definition():
        o, b = np.zeros((4, Hq, d)), np.zeros((4, Hq, d))
        for n in range(4):
            where = np.array([int(prefix[j // page]) for j in left] + [int(table[n, j // page]) for j in range(lens[n])])
            rows = np.array([j % page for j in left] + [j % page for j in range(lens[n])])
            for h in range(Hq):
                y, s, r = oa.row(np64(q)[n, h], np64(kc)[where, h // (Hq // Hk), rows], np64(vc)[where, h // (Hq // Hk), rows],
                                 d ** -0.5)
                o[n, h] = y
                b[n, h] = oa.attention_bound(y, s, np.array(r), 256, d, BITS[dtype], 8 if dtype == BF16 else None)
        return o, b
    run = lambda: np64(lr.lr_step_paged_prefix(q.to(dev), kc, vc, broken, P, wider(table, max_len, page, dev),
                                               torch.tensor(lens, dtype=torch.int32, device=dev), max_len=max_len))
    want, bound = definition()
    vc[place(prefix, 9)][:, 3], vc[place(prefix, 100)][:, 5], vc[place(prefix, 101)][:, 6] = inf, -inf, nan
    vc[place(table[1], 0)][:, 5], vc[place(table[3], 32)][:, 7] = inf, -inf
    vc[place(prefix, 40)] = nan      # on the page that is left out
    got = run()
    assert lr.device_status() == LR_ERR_INDEX
    for n in range(4):
        for ch, x in ((3, inf), (5, nan if n == 1 else -inf), (6, nan)) + (((7, -inf),) if n == 3 else ()):
            assert np.array_equal(got[n, :, ch], np.full(Hq, x), equal_nan=True), (n, ch, got[n, :, ch])
            got[n, :, ch] = want[n, :, ch] = 0
    within(torch.from_numpy(got), want, bound)
    for j in range(P):
        vc[place(prefix, j)] = torch.finfo(dtype).max / 2
    for n in range(4):
        for j in range(lens[n]):
            vc[place(table[n], j)] = torch.finfo(dtype).max / 2
    got = run()
    assert lr.device_status() == LR_ERR_INDEX
    within(torch.from_numpy(got / np64(torch.finfo(dtype).max * torch.ones(()))), np.full_like(got, 0.5),
           2.0 ** -BITS[dtype] + 2.0 ** -16)


@types
@pytest.mark.parametrize("top", [2.0 ** 33, 2.0 ** 66, 2.0 ** 126], ids=str)
@pytest.mark.parametrize("where", ["prefix", "own"])
def test_prefix_large_finite_scores(dev, where, top, dtype):
    """Scores of 1e10 and more: those alike share the weight between prefix and
    own tokens, one a 64th part above them takes all of it."""
    d, P, lens, page = 64, 300, [40, 40], 16
    kc, vc, prefix, table = shared(91, P, lens, 1, page, d, dtype, dev)
    q = torch.zeros(2, 2, d, dtype=dtype)
    q[..., 0] = 1
    kc.zero_()
    kc[..., 0] = torch.tensor(top * (1 - 2.0 ** -6))
    args = (prefix, P, table, torch.tensor(lens, dtype=torch.int32, device=dev))
    o = lr.lr_step_paged_prefix(q.to(dev), kc, vc, *args, scale=1.0)
    ref, size, reach, _ = oa.step_prefix(np64(q), np64(kc), np64(vc), prefix.cpu().numpy(), P, table.cpu().numpy(), lens,
                                         NW, 0, 1.0)
    # products with 0 and 1 are exact, so the scores are: reach 0
    bound = oa.attention_bound(ref, size, np.zeros_like(reach), 340, d, BITS[dtype], 8 if dtype == BF16 else None)
    within(o, ref, bound)
    pages, j = (prefix, 170) if where == "prefix" else (table[0], 20)
    kc[int(pages[j // page]), 0, j % page, 0] = top
    o = lr.lr_step_paged_prefix(q.to(dev), kc, vc, *args, scale=1.0)
    alone = vc[int(pages[j // page]), 0, j % page]
    rows = o if where == "prefix" else o[:1]
    # fp32 values enter the products as two parts of 11 bits: 2^-22 of a value is
    # left out, and the result rounded once; bf16 values are exact
    want = np.broadcast_to(np64(alone), rows.shape)
    within(rows, want, np.abs(want) * (2.0 ** -22 + 2.0 ** -24 if dtype == F32 else 0.0))


@types
@pytest.mark.parametrize("base", [1.8125, 1.46875, -1.8125])
def test_prefix_weights_of_parts_agree_at_large_scores(dev, base, dtype):
    """512 keys of the prefix at a score of some 2^21, one own key 7 above them:
    both parts refer to the same maximum.  Scores are exact, and what the
    exponential takes is below 32, so its roundings are those of scores of that
    size."""
    d, P, page, lens = 64, 512, 64, [1, 1]
    kc, vc, prefix, table = shared(95, P, lens, 1, page, d, dtype, dev)
    q = torch.zeros(2, 1, d, dtype=dtype)
    q[..., :2] = 1
    kc.zero_()
    kc[..., 0] = base * 2.0 ** 21
    vc.fill_(1.0)
    for n in range(2):
        kc[int(table[n, 0]), 0, 0, 1] = 7.0
        vc[int(table[n, 0]), 0, 0] = -1
    o = lr.lr_step_paged_prefix(q.to(dev), kc, vc, prefix, P, table, torch.tensor(lens, dtype=torch.int32, device=dev),
                                scale=1.0)
    ref, size, reach, _ = oa.step_prefix(np64(q), np64(kc), np64(vc), prefix.cpu().numpy(), P, table.cpu().numpy(), lens,
                                         NW, 0, 1.0)
    bound = oa.attention_bound(ref, size, np.full_like(reach, 32.0), 513, d, BITS[dtype], 8 if dtype == BF16 else None)
    within(o, ref, bound)


@types
@pytest.mark.parametrize("which", ["k", "v"])
def test_prefix_full_of_nan_stays_quick(dev, which, dtype):
    import time
    N, P, page, d = 64, 4096, 64, 64
    kc, vc = (rnd(s, 64 + N, 2, page, d, dtype=dtype).to(dev) for s in (1, 2))
    (kc if which == "k" else vc).fill_(float("nan"))
    prefix = torch.arange(64, dtype=torch.int32, device=dev)
    table = torch.arange(64, 64 + N, dtype=torch.int32, device=dev)[:, None].contiguous()
    q, lens = rnd(3, N, 8, d, dtype=dtype).to(dev), torch.full((N,), 60, dtype=torch.int32, device=dev)
    lr.lr_step_paged_prefix(q, kc, vc, prefix, P, table, lens)
    torch.cuda.synchronize()
    t0 = time.time()
    o = lr.lr_step_paged_prefix(q, kc, vc, prefix, P, table, lens)
    torch.cuda.synchronize()
    assert time.time() - t0 < 0.5
    assert o.isnan().all()


@types
def test_prefix_bad_pages_and_lengths_are_reported(dev, dtype):
    """A page of the prefix outside the pool is left out for all sequences, one of
    a sequence for it alone; a length beyond the bound leaves its row as it was."""
    lens, d, page, P = [40, 40, 40], 64, 16, 100
    kc, vc, prefix, table = shared(8, P, lens, 1, page, d, dtype, dev)
    q = rnd(34, 3, 2, d, dtype=dtype)
    ld = torch.tensor(lens, dtype=torch.int32, device=dev)
    step = lambda pages, t, n=ld, **kw: lr.lr_step_paged_prefix(q.to(dev), kc, vc, pages, P, t, n, **kw)
    good = step(prefix, table)
    assert lr.device_status() == LR_OK
    for bad in (-1, kc.shape[0], 2 ** 31 - 1, -2 ** 31):
        broken = table.clone()
        broken[1, 2] = bad
        o = step(prefix, broken)
        assert lr.device_status() == LR_ERR_INDEX and lr.device_status() == LR_OK
        assert torch.equal(o[0], good[0]) and torch.equal(o[2], good[2]) and o.isfinite().all()
        broken = prefix.clone()
        broken[3] = bad
        o = step(broken, table)
        assert lr.device_status() == LR_ERR_INDEX and lr.device_status() == LR_OK
        # the same keys without that page: a prefix of 84 tokens
        rest = torch.cat((prefix[:3], prefix[4:]))
        ref, size, reach, _ = oa.step_prefix(np64(q), np64(kc), np64(vc), rest.cpu().numpy(), P - page,
                                             table.cpu().numpy(), lens, NW, 0, d ** -0.5)
        within(o, ref, oa.attention_bound(ref, size, reach, 140, d, BITS[dtype], 8 if dtype == BF16 else None))
    o = torch.full_like(good, 7.0)
    step(prefix, table, torch.tensor([40, 41, 2 ** 31 - 1], dtype=torch.int32, device=dev), max_len=40, o=o)
    assert lr.device_status() == LR_ERR_INDEX
    assert torch.equal(o[0], good[0]) and (o[1:] == 7).all()


@types
def test_prefix_offsets_past_32_bits(dev, dtype):
    """The last pages of a pool of more than 2^31 elements."""
    Hk, page, d, P, lens = 2, 256, 128, 600, [300]
    total = (1 << 31) // (Hk * page * d) + 6
    kc, vc, prefix, table = shared(9, P, lens, Hk, page, d, dtype, dev)
    big = [torch.empty(total, Hk, page, d, dtype=dtype, device=dev) for _ in range(2)]
    moved = [prefix.clone(), table.clone()]
    at = total
    for pages in (moved[0], moved[1][0]):
        for j in range(len(pages)):
            at -= 1
            big[0][at], big[1][at] = kc[int(pages[j])], vc[int(pages[j])]
            pages[j] = at
    q = rnd(35, 1, 4, d, dtype=dtype).to(dev)
    ld = torch.tensor(lens, dtype=torch.int32, device=dev)
    assert torch.equal(lr.lr_step_paged_prefix(q, *big, moved[0], P, moved[1], ld),
                       lr.lr_step_paged_prefix(q, kc, vc, prefix, P, table, ld))


@types
def test_prefix_captures_into_graphs_that_share_a_workspace(dev, dtype):
    """Replays follow queries and lengths; two graphs use one workspace in turn."""
    N, Hq, Hk, d, page, P, most = 5, 4, 1, 64, 16, 1000, 400
    kc, vc = (rnd(s, 63 + N * most, Hk, page, d, dtype=dtype).to(dev) for s in (60, 61))
    prefix = torch.arange(63, dtype=torch.int32, device=dev)
    table = (63 + torch.arange(N * most, device=dev)).int().view(N, most)
    q = rnd(62, N, Hq, d, dtype=dtype).to(dev)
    lens = torch.tensor([5901, 5, 0, 70, 300], dtype=torch.int32, device=dev)
    need = max(lr.step_paged_prefix_workspace_size(N, Hq, Hk, d, P, most * page, dtype, w) for w in (None, 700))
    ws = torch.empty(need, dtype=torch.uint8, device=dev)
    once = lambda window: lr.lr_step_paged_prefix(q, kc, vc, prefix, P, table, lens, window=window, workspace=ws)
    once(None), once(700)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for window in (None, 700):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(once(window))
        graphs.append(g)
    for s in range(3):
        q.copy_(rnd(63 + s, *q.shape, dtype=dtype))
        for i, window in ((0, None), (1, 700), (0, None)):
            outs[i].fill_(7.0)
            graphs[i].replay()
            assert torch.equal(outs[i], once(window))
        lens += 1


@types
def test_prefix_two_calls_at_once_and_another_stream(dev, dtype):
    P, lens = 3000, [400, 40, 300]
    kc, vc, prefix, table = shared(11, P, lens, 2, 64, 128, dtype, dev)
    q, ld = rnd(70, 3, 8, 128, dtype=dtype).to(dev), torch.tensor(lens, dtype=torch.int32, device=dev)
    want = [lr.lr_step_paged_prefix(q, kc, vc, prefix, P, table, ld, window=w) for w in (None, 500)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(dev) for _ in range(2)]
    for _ in range(3):
        got = [lr.lr_step_paged_prefix(q, kc, vc, prefix, P, table, ld, window=w, stream=s)
               for s, w in zip(streams, (None, 500))]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@types
@pytest.mark.parametrize("max_len", CUTS)
def test_prefix_calls_in_a_row_on_one_workspace(dev, max_len, dtype):
    """The own tokens' kernel may start under the prefix's last CTAs: calls that
    follow each other without a pause, some with no sequence at all, some with new
    queries and lengths written just before, give what single calls give."""
    P, d, page, tries = 1500, 64, 64, 12
    kc, vc, prefix, table = shared(140, P, [64] * 6, 2, page, d, dtype, dev)
    table = wider(table, max_len, page, dev)
    qs = [rnd(141 + i, 6, 4, d, dtype=dtype).to(dev) for i in range(tries)]
    r = np.random.RandomState(3)
    lens = [torch.tensor(r.randint(0, 65, 6) if i % 4 else [-1] * 6, dtype=torch.int32, device=dev) for i in range(tries)]
    ws = torch.empty(lr.step_paged_prefix_workspace_size(6, 4, 2, d, P, max_len, dtype), dtype=torch.uint8, device=dev)
    call = lambda q, ld: lr.lr_step_paged_prefix(q, kc, vc, prefix, P, table, ld, max_len=max_len, workspace=ws)
    want = []
    for q, ld in zip(qs, lens):
        want.append(call(q, ld))
        torch.cuda.synchronize()
        ws.fill_(255)
    q, ld, got = qs[0].clone(), lens[0].clone(), []
    for i in range(tries):
        q.copy_(qs[i])
        ld.copy_(lens[i])
        got.append(call(q, ld))
        if i % 3 == 2:
            ws.fill_(255)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@types
@pytest.mark.parametrize("N", [123, 256, 257])
def test_prefix_batches_taken_by_length(dev, N, dtype):
    """More CTAs than run at once: the longest sequences come first, equal lengths,
    empty and unused slots among them; beyond 256 sequences in their order."""
    Hk, d, page, P = 5, 32, 16, 70
    lens = np.random.RandomState(N).choice([-1, 0, 1, 7, 16, 40, 40, 61], N)
    lens[[0, N // 2, N - 1]] = 61, -1, 33
    kc, vc, prefix, table = shared(160, P, lens.tolist(), Hk, page, d, dtype, dev)
    check(dev, rnd(161, N, 2 * Hk, d, dtype=dtype), kc, vc, prefix, P, table, lens.tolist(), NW, 0)
    check(dev, rnd(162, N, 2 * Hk, d, dtype=dtype), kc, vc, prefix, P, table, lens.tolist(), 50, 3)


@types
def test_prefix_pages_held_more_than_once(dev, dtype):
    """A page twice in the prefix, the prefix's pages among the own ones, the same
    own pages for several sequences."""
    d, page, P, lens = 128, 16, 70, [40, 40, 17, 33]
    kc, vc = (rnd(s, 9, 2, page, d, dtype=dtype).to(dev) for s in (150, 151))
    prefix = torch.tensor([4, 1, 4, 0, 7], dtype=torch.int32, device=dev)
    table = torch.tensor([[4, 0, 8], [4, 0, 8], [2, 2, 2], [8, 1, 3]], dtype=torch.int32, device=dev)
    check(dev, rnd(152, 4, 6, d, dtype=dtype), kc, vc, prefix, P, table, lens, NW, 0)
    check(dev, rnd(153, 4, 6, d, dtype=dtype), kc, vc, prefix, P, table, lens, 60, 20)


@types
def test_prefix_then_sequences_of_their_own(dev, dtype):
    """A prefix written once by the rotation's append, then a few tokens of each
    sequence one by one: every row is that of the whole sequence under
    lr_fwd_window."""
    N, P, more, Hq, Hk, d, page, window, sinks = 3, 150, 4, 4, 2, 64, 16, 120, 5
    f = torch.tensor(10000.0 ** (-np.arange(d // 2) / (d // 2)), device=dev)
    x = rnd(80, 1, P, Hq + 2 * Hk, d, dtype=dtype).to(dev)
    own = rnd(81, N, more, Hq + 2 * Hk, d, dtype=dtype).to(dev)
    prefix = torch.arange(10, dtype=torch.int32, device=dev)
    table = torch.arange(10, 10 + N, dtype=torch.int32, device=dev)[:, None].contiguous()
    kc, vc = (torch.zeros(10 + N, Hk, page, d, dtype=dtype, device=dev) for _ in range(2))
    cut = ((0, Hq), (Hq, Hq + Hk), (Hq + Hk, Hq + 2 * Hk))
    split = lambda t: [t[:, :, i:j].transpose(1, 2) for i, j in cut]
    q, k, v = split(x)
    _, k0 = lr.lr_qk_norm_rope(q, k, inv_freq=f, v=v, k_cache=kc, v_cache=vc, table=prefix[None])
    keys, values, queries, got = [k0.expand(N, -1, -1, -1)], [v.expand(N, -1, -1, -1)], [], []
    axis = torch.zeros(d // 2, dtype=torch.int32, device=dev)
    for t in range(more):
        q, k, v = split(own[:, t:t + 1])
        # positions of the whole sequence, the cache row among the own tokens
        at, place = (torch.full((N, 1), n, dtype=torch.int32, device=dev) for n in (P + t, t))
        qo, ko = lr.lr_qk_norm_rope_axes(q, k, at[None], axis, place, inv_freq=f, v=v, k_cache=kc, v_cache=vc, table=table)
        lens = torch.full((N,), t + 1, dtype=torch.int32, device=dev)
        got.append(lr.lr_step_paged_prefix(qo[:, :, 0].contiguous(), kc, vc, prefix, P, table, lens, window=window,
                                           sinks=sinks)[:, :, None])
        keys.append(ko), values.append(v), queries.append(qo)
    q, k, v = (torch.cat(t, 2) for t in (queries, keys, values))
    ref, size, reach, _ = oa.window(np64(q), np64(k), np64(v), window, sinks, d ** -0.5)
    bound = oa.attention_bound(ref, size, reach, P + more, d, BITS[dtype], 8 if dtype == BF16 else None)
    within(torch.cat(got, 2), ref, bound)
