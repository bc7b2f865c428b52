"""lr_step_paged_diff against its fp64 definition (oracle/attention.py), element
by element within the bound derived there; and prompts and steps together.
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
EPS = 1e-6
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
    kc, vc = (torch.full((total, 2 * Hk, page, d), float("nan"), dtype=dtype) for _ in range(2))
    at = 0
    for n, L in enumerate(lens):
        for j in range(need[n]):
            pg = int(order[at])
            at += 1
            table[n, j] = pg
            rows = min(page, L - j * page)
            kc[pg, :, :rows] = rnd(seed + 31 * at, 2 * Hk, rows, d, dtype=dtype)
            vc[pg, :, :rows] = rnd(seed + 31 * at + 7, 2 * Hk, rows, d, dtype=dtype)
    return kc.to(dev), vc.to(dev), torch.from_numpy(table).to(dev)


def wider(table, max_len, page, dev):
    wide = torch.zeros(table.shape[0], -(-max_len // page), dtype=torch.int32, device=dev)
    most = min(wide.shape[1], table.shape[1])
    wide[:, :most] = table[:, :most]
    return wide


def check(dev, q, kc, vc, table, lens, lam, window, sinks, scale=None, max_len=None, norm=True, weight=None):
    dtype, d = q.dtype, q.shape[-1]
    scale = d ** -0.5 if scale is None else scale
    o = torch.full(q.shape, 7.0, dtype=dtype, device=dev)
    ld = torch.tensor(lens, dtype=torch.int32, device=dev)
    args = dict(max_len=max_len, window=window, sinks=sinks, scale=scale, norm=norm, eps=EPS,
                norm_weight=None if weight is None else weight.to(dev))
    out = lr.lr_step_paged_diff(q.to(dev), kc, vc, table, ld, lam.to(dev), o=o, **args)
    torch.cuda.synchronize()
    assert out is o
    ref, bound, written = oa.diff_step(np64(q), np64(kc), np64(vc), table.cpu().numpy(), lens, np64(lam), window, sinks,
                                       scale, BITS[dtype], 8 if dtype == BF16 else None,
                                       None if weight is None else np64(weight), EPS if norm else None)
    w = np.broadcast_to(written[:, None, None], ref.shape)
    within(out, np.where(w, ref, 7.0), np.where(w, bound, 0.0))
    made = lr.lr_step_paged_diff(q.to(dev), kc, vc, table, ld, lam.to(dev), **args)
    assert torch.equal(made, torch.where(torch.from_numpy(w.copy()).to(dev), out, torch.zeros_like(out)))
    return out


def lams(H, seed=0):
    return 0.2 + 0.6 * torch.rand(H, generator=torch.Generator().manual_seed(seed))


LENS = [1, 0, 15, 16, 17, -1, 127, 128, 129, 300, 601]


@types
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("H,Hk", [(1, 1), (4, 2), (3, 1), (9, 1), (6, 6)])
@pytest.mark.parametrize("page,window,sinks", [(16, NW, 0), (64, 40, 5), (128, 130, 20)])
def test_diff_step_parity(dev, dtype, d, H, Hk, page, window, sinks):
    """Lengths of zero, one, page and chunk edges; unused slots; NaN in every
    row of the pools that no sequence holds."""
    kc, vc, table = paged(d + H, LENS, Hk, page, d, dtype, dev)
    check(dev, rnd(30, len(LENS), 2 * H, d, dtype=dtype), kc, vc, table, LENS, lams(H), window, sinks,
          weight=rnd(29, 2 * d) if H > 1 else None)


@types
@pytest.mark.parametrize("norm", [True, False], ids=["norm", "plain"])
@pytest.mark.parametrize("d", [32, 128])
@pytest.mark.parametrize("max_len,window,sinks", [(64, NW, 0), (65, NW, 0), (700, NW, 0), (4097, NW, 0), (40000, NW, 0),
                                                  (20000, 300, 0), (20000, 300, 7), (20000, 4000, 64)])
def test_diff_step_cut_by_the_bound_on_the_length(dev, dtype, d, norm, max_len, window, sinks):
    lens = [x for x in (1, 0, 64, -1, 63, 700, 4096, 7000) if x <= max_len]
    kc, vc, table = paged(21, lens, 2, 64, d, dtype, dev)
    check(dev, rnd(37, len(lens), 6 * 2, d, dtype=dtype), kc, vc, wider(table, max_len, 64, dev), lens, lams(6), window,
          sinks, max_len=max_len, norm=norm)


@types
@pytest.mark.parametrize("d,H,Hk", [(32, 8, 8), (128, 8, 2), (64, 9, 1)])
@pytest.mark.parametrize("N", [3, 6, 8, 9, 13, 19, 38])
def test_diff_step_cluster_sizes(dev, dtype, d, H, Hk, N):
    lens = [(1500 - 41 * i) % 1501 for i in range(N)]
    kc, vc, table = paged(N, lens, Hk, 64, d, dtype, dev)
    check(dev, rnd(52, N, 2 * H, d, dtype=dtype), kc, vc, table, lens, lams(H), NW, 0)


@types
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (16, 3), (33, 50), (250, 17), (NW, 4)])
@pytest.mark.parametrize("page", [16, 256])
def test_diff_step_sees_each_key_once(dev, dtype, window, sinks, page):
    d, lens = 128, [290, 31, 257]
    kc, vc, table = paged(3, lens, 1, page, d, dtype, dev)
    for n, L in enumerate(lens):
        for j in range(L):
            pg = int(table[n, j // page])
            kc[pg, :, j % page] = 0
            vc[pg, :, j % page] = 0
            vc[pg, (j // d) % 2, j % page, j % d] = 1
    check(dev, rnd(31, 3, 4, d, dtype=dtype), kc, vc, table, lens, lams(2), window, sinks, 1.0, norm=False)


@types
@pytest.mark.parametrize("max_len", CUTS)
@pytest.mark.parametrize("scale", [0.0, -0.4, 1e-3])
def test_diff_step_scales(dev, dtype, scale, max_len):
    lens = [64, 3, 50]
    kc, vc, table = paged(22, lens, 1, 16, 64, dtype, dev)
    check(dev, rnd(23, 3, 4, 64, dtype=dtype), kc, vc, wider(table, max_len, 16, dev), lens, torch.tensor([0.4, -0.9]), NW,
          0, scale, max_len=max_len, norm=scale != 0.0)


@types
def test_diff_step_masked_keys_may_hold_anything(dev, dtype):
    lens, d, page = [400, 131], 128, 32
    kc, vc, table = paged(6, lens, 2, page, d, dtype, dev)
    clean_k, clean_v = kc.clone(), vc.clone()
    for n, L in enumerate(lens):
        for j in range(5, L - 100):
            kc[int(table[n, j // page]), :, j % page] = float("nan") if j % 2 else float("inf")
            vc[int(table[n, j // page]), :, j % page] = float("inf") if j % 3 else float("nan")
    q = rnd(33, 2, 8, d, dtype=dtype)
    a = check(dev, q, kc, vc, table, lens, lams(4), 100, 5)
    b = check(dev, q, clean_k, clean_v, table, lens, lams(4), 100, 5)
    assert torch.equal(a, b)


@types
@pytest.mark.parametrize("d,H,Hk", [(32, 2, 1), (64, 9, 1), (128, 6, 2)])
@pytest.mark.parametrize("max_len", CUTS)
def test_diff_step_seen_infinities_and_nan(dev, max_len, d, H, Hk, dtype):
    """As over whole sequences: a seen infinity is NaN where lambda is positive
    and that infinity where it is negative, a NaN stays in its channel, a NaN key
    makes its pairs NaN; with the norm other channels are 0 or NaN.  A page outside
    the pool is left out of all this."""
    page, inf, nan, lens = 16, float("inf"), float("nan"), [50, 61, 33, 64]
    kc, vc, table = paged(130, lens, Hk, page, d, dtype, dev)
    q = rnd(131, len(lens), 2 * H, d, dtype=dtype)
    lam = lams(H)
    lam[0::2] *= -1
    ref, bound, _ = oa.diff_step(np64(q), np64(kc), np64(vc), table.cpu().numpy(), lens, np64(lam), NW, 0, d ** -0.5,
                                 BITS[dtype], 8 if dtype == BF16 else None)
    # sequence 3: its second page is outside the pool
    left = np.array([j for j in range(lens[3]) if j // page != 1])
    where, rows = table[3].cpu().numpy()[left // page], left % page
    for h in range(H):
        g = h // (H // Hk)
        k = [np64(kc)[where, 2 * g + m, rows] for m in range(2)]
        v = np.concatenate([np64(vc)[where, 2 * g + m, rows] for m in range(2)], -1)
        y, e = oa.diff_rows(np64(q)[3, 2 * h][None], np64(q)[3, 2 * h + 1][None], *k, v, np.ones((1, len(left)), bool),
                            d ** -0.5, float(lam[h]), d, BITS[dtype], 8 if dtype == BF16 else None)
        ref[3, 2 * h:2 * h + 2], bound[3, 2 * h:2 * h + 2] = y.reshape(2, d), e.reshape(2, d)
    place = lambda n, j: (int(table[n, j // page]), slice(None), j % page)
    vc[place(0, 9)][0::2, 3] = inf       # channel 3 of the first halves
    vc[place(1, 60)][1::2, 5] = nan      # channel 5 of the second halves
    kc[place(2, 32)][0::2, 1] = nan      # the keys of map 0
    vc[place(3, 20)] = nan               # on the page that is left out
    wide = wider(table, max_len, page, dev)
    wide[3, 1] = kc.shape[0]
    need = lr.step_paged_diff_workspace_size(len(lens), H, Hk, d, max_len, dtype)
    assert (need > 0) == (max_len == CUTS[2])
    run = lambda norm: lr.lr_step_paged_diff(q.to(dev), kc, vc, wide, torch.tensor(lens, dtype=torch.int32, device=dev),
                                             lam.to(dev), max_len=max_len, norm=norm, eps=EPS)
    got = np64(run(False))
    assert lr.device_status() == LR_ERR_INDEX
    want = np.where(np64(lam) < 0, inf, nan)
    assert np.array_equal(got[0, 0::2, 3], want, equal_nan=True)
    assert np.isnan(got[1, 1::2, 5]).all() and np.isnan(got[2]).all()
    for n, half, ch in ((0, 0, 3), (1, 1, 5)):
        got[n, half::2, ch] = ref[n, half::2, ch] = 0
    got[2] = ref[2] = 0
    within(torch.from_numpy(got), ref, 2 * bound)
    normed = np64(run(True))
    assert lr.device_status() == LR_ERR_INDEX
    assert np.isnan(normed[1:3]).all() and np.isfinite(normed[3]).all()
    for h in range(H):
        row = normed[0, 2 * h:2 * h + 2].reshape(-1)
        if lam[h] > 0:
            assert np.isnan(row).all()
        else:
            assert np.isnan(row[3]) and (np.delete(row, 3) == 0).all()


@types
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("max_len", CUTS)
def test_diff_step_values_at_the_end_of_the_type(dev, max_len, d, dtype):
    """Means of the type's largest values do not overflow; with the norm their
    squares do, and the row is divided by infinity."""
    lens = [64, 37]
    kc, vc, table = paged(132, lens, 1, 16, d, dtype, dev)
    vc.fill_(torch.finfo(dtype).max)
    lam = torch.tensor([0.5, 0.25], device=dev)
    args = (rnd(133, 2, 4, d, dtype=dtype).to(dev), kc, vc, wider(table, max_len, 16, dev),
            torch.tensor(lens, dtype=torch.int32, device=dev), lam)
    o = np64(lr.lr_step_paged_diff(*args, max_len=max_len, norm=False)) / float(torch.finfo(dtype).max)
    for h, x in enumerate((0.5, 0.75)):
        assert (np.abs(o[:, 2 * h:2 * h + 2] - x) <= (2.0 ** -7 if dtype == BF16 else 2.0 ** -14)).all()
    assert (lr.lr_step_paged_diff(*args, max_len=max_len) == 0).all()


@types
def test_diff_step_bad_pages_and_lengths_are_reported(dev, dtype):
    lens, d, page = [40, 40, 40], 64, 16
    kc, vc, table = paged(8, lens, 1, page, d, dtype, dev)
    q, lam = rnd(34, 3, 4, d, dtype=dtype).to(dev), lams(2).to(dev)
    ld = torch.tensor(lens, dtype=torch.int32, device=dev)
    for bound_on_len in (40, 300, 20000):
        wide = wider(table, max(bound_on_len, 48), page, dev)
        good = lr.lr_step_paged_diff(q, kc, vc, wide, ld, lam, max_len=bound_on_len)
        assert lr.device_status() == LR_OK
        for bad in (-1, kc.shape[0], 2 ** 31 - 1, -2 ** 31):
            broken = wide.clone()
            broken[1, 2] = bad
            o = lr.lr_step_paged_diff(q, kc, vc, broken, ld, lam, max_len=bound_on_len)
            assert lr.device_status() == LR_ERR_INDEX and lr.device_status() == LR_OK
            assert torch.equal(o[0], good[0]) and torch.equal(o[2], good[2]) and o.isfinite().all()
        o = torch.full_like(q, 7.0)
        lr.lr_step_paged_diff(q, kc, vc, wide, torch.tensor([40, bound_on_len + 1, 2 ** 31 - 1], dtype=torch.int32, device=dev),
                              lam, max_len=bound_on_len, o=o)
        assert lr.device_status() == LR_ERR_INDEX
        assert torch.equal(o[0], good[0]) and (o[1:] == 7).all()


@types
def test_diff_step_offsets_past_32_bits(dev, dtype):
    """The last pages of a pool of more than 2^31 elements."""
    Hk, page, d = 1, 256, 128
    total = (1 << 31) // (2 * Hk * page * d) + 3
    lens = [520]
    kc, vc, table = paged(9, lens, Hk, page, d, dtype, dev)
    big = [torch.empty(total, 2 * Hk, page, d, dtype=dtype, device=dev) for _ in range(2)]
    moved = table.clone()
    for j in range(3):
        moved[0, j] = total - 1 - j
        big[0][total - 1 - j], big[1][total - 1 - j] = kc[int(table[0, j])], vc[int(table[0, j])]
    q, lam = rnd(35, 1, 4, d, dtype=dtype).to(dev), lams(2).to(dev)
    ld = torch.tensor(lens, dtype=torch.int32, device=dev)
    assert torch.equal(lr.lr_step_paged_diff(q, *big, moved, ld, lam), lr.lr_step_paged_diff(q, kc, vc, table, ld, lam))


@types
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("window,sinks", [(24, 3), (None, 0)])
def test_prompt_then_steps_together(dev, dtype, d, window, sinks):
    """A prompt with positions of three axes through rotation and append,
    attention, then its next tokens one by one over the pages: every row is that of
    the whole sequence."""
    B, T, more, H, Hk, page = 2, 70, 5, 4, 2, 16
    total = T + more
    f = torch.tensor(10000.0 ** (-np.arange(d // 2) / (d // 2)), device=dev)
    axis = (torch.arange(d // 2, device=dev) % 3).int()
    r = np.random.RandomState(4)
    pos = r.randint(0, 90, (3, B, total)).astype(np.int32)
    x = rnd(80, B, total, 2 * H + 4 * Hk, d, dtype=dtype)
    cut = ((0, 2 * H), (2 * H, 2 * H + 2 * Hk), (2 * H + 2 * Hk, 2 * H + 4 * Hk))
    table = torch.from_numpy(r.permutation(2 * 5).reshape(2, 5).astype(np.int32)).to(dev)
    kc, vc = (torch.zeros(10, 2 * Hk, page, d, dtype=dtype, device=dev) for _ in range(2))
    lam, weight = lams(H), rnd(81, 2 * d)
    outs, keys, queries = [], [], []
    xd = x.to(dev)
    for a, b in [(0, T)] + [(t, t + 1) for t in range(T, total)]:
        q, k, v = (xd[:, a:b, i:j].transpose(1, 2) for i, j in cut)
        place = torch.arange(a, b, dtype=torch.int32, device=dev).expand(B, b - a).contiguous()
        qo, ko = lr.lr_qk_norm_rope_axes(q, k, torch.from_numpy(pos[:, :, a:b].copy()).to(dev), axis, place, inv_freq=f,
                                         v=v, k_cache=kc, v_cache=vc, table=table)
        keys.append(ko), queries.append(qo)
        args = dict(window=window, sinks=sinks, norm_weight=weight.to(dev), eps=EPS)
        if a == 0:
            outs.append(lr.lr_fwd_diff(qo, ko, v, lam.to(dev), **args))
        else:
            lens = torch.full((B,), b, dtype=torch.int32, device=dev)
            outs.append(lr.lr_step_paged_diff(qo[:, :, 0].contiguous(), kc, vc, table, lens, lam.to(dev), **args)[:, :, None])
    q, k = torch.cat(queries, 2), torch.cat(keys, 2)
    v = x[:, :, cut[2][0]:].transpose(1, 2)
    ref, bound, _ = oa.diff(np64(q), np64(k), np64(v), np64(lam), NW if window is None else window, sinks, d ** -0.5,
                            BITS[dtype], 8 if dtype == BF16 else None, np64(weight), EPS)
    within(torch.cat(outs, 2), ref, bound)


def test_diff_step_captures_into_graphs_that_share_a_workspace(dev):
    B, H, Hk, d, page, most = 2, 4, 1, 128, 16, 400
    table = torch.arange(B * most, dtype=torch.int32, device=dev).view(B, most)
    kc, vc = (rnd(s, B * most, 2 * Hk, page, d, dtype=BF16).to(dev) for s in (60, 61))
    q, lam = rnd(62, B, 2 * H, d, dtype=BF16).to(dev), lams(H).to(dev)
    lens = torch.tensor([5901, 5], dtype=torch.int32, device=dev)
    ws = torch.empty(lr.step_paged_diff_workspace_size(B, H, Hk, d, most * page, BF16), dtype=torch.uint8, device=dev)
    assert ws.numel() > 0
    once = lambda window: lr.lr_step_paged_diff(q, kc, vc, table, lens, lam, window=window, workspace=ws)
    once(None), once(700)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for window in (None, 700):   # chunks joined by a kernel, and by a cluster
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(once(window))
        graphs.append(g)
    for s in range(3):
        q.copy_(rnd(63 + s, *q.shape, dtype=BF16))
        lam.mul_(0.9)
        for i, window in ((0, None), (1, 700), (0, None)):
            outs[i].fill_(7.0)
            graphs[i].replay()
            assert torch.equal(outs[i], once(window))
        lens += 1


@types
def test_diff_step_two_calls_at_once_and_another_stream(dev, dtype):
    lens = [4000, 40, 3000]
    kc, vc, table = paged(11, lens, 2, 64, 64, dtype, dev)
    q, lam, ld = rnd(70, 3, 8, 64, dtype=dtype).to(dev), lams(4).to(dev), torch.tensor(lens, dtype=torch.int32, device=dev)
    want = [lr.lr_step_paged_diff(q, kc, vc, table, ld, lam, window=w) for w in (None, 500)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(dev) for _ in range(2)]
    for _ in range(3):
        got = [lr.lr_step_paged_diff(q, kc, vc, table, ld, lam, window=w, stream=s) for s, w in zip(streams, (None, 500))]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
