"""lr_fwd_diff: long rows, rows beside values that are not finite, and what the
weights' and the squares' range leave, against the fp64 definition."""
import numpy as np
import pytest
import torch

import gated_delta_rule_fwd_gb300 as lr
from oracle import attention as oa

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
BITS = {F32: 24, BF16: 8}          # half a step of the type, 2^-bits relative
NW = lr.NO_WINDOW
LR_OK = 0
EPS = 1e-6
types = pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
widths = pytest.mark.parametrize("d", [32, 64, 128])


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


def within(got, want, bound, what=""):
    got = np64(got)
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} outside, first at {np.argwhere(bad)[0]}: "
                           f"{got[bad][0]} for {want[bad][0]} +- {bound[bad][0]}")


def inputs(B, H, Hk, Tq, Tk, d, dtype, seed=1):
    q, k, v = (rnd(seed + i, B, 2 * h, t, d, dtype=dtype) for i, (h, t) in enumerate(((H, Tq), (Hk, Tk), (Hk, Tk))))
    return q, k, v, 0.2 + 0.6 * torch.rand(H, generator=torch.Generator().manual_seed(seed))


@types
@widths
def test_diff_rows_of_many_tiles(dev, d, dtype):
    """Rows over up to 32 tiles, whose maxima grow along the way, so that scores, weights and
    outputs are rescaled and replaced in turn: right, and the same bits each time."""
    H, T = 2, 4096
    q, k, v, lam = inputs(1, H, 1, T, T, d, dtype, seed=301)
    k = (k.float() * torch.linspace(0.1, 3.0, T)[:, None]).to(dtype)
    ref, bound, _ = oa.diff(np64(q), np64(k), np64(v), np64(lam), NW, 0, d ** -0.5, BITS[dtype],
                            8 if dtype == BF16 else None, None, EPS)
    on = [t.to(dev) for t in (q, k, v, lam)]
    first = lr.lr_fwd_diff(*on, eps=EPS)
    within(first, ref, bound)
    for _ in range(20):
        assert torch.equal(lr.lr_fwd_diff(*on, eps=EPS), first)


LONG = 8192


def _seconds(call):
    import time
    torch.cuda.synchronize()
    t0 = time.time()
    o = call()
    torch.cuda.synchronize()
    return o, time.time() - t0


@widths
@pytest.mark.parametrize("norm", [True, False], ids=["norm", "plain"])
def test_diff_one_early_infinity_in_a_long_sequence(dev, norm, d):
    """Every row but the first few sees an infinity in one channel, none has an end in
    sight before its last key: all rows are written, in time, and no wait gives up.
    Without the norm that channel is NaN where lambda is positive and the infinity where
    it is negative, and the others are as without it; with the norm NaN in all channels
    or in that one, with zeros beside it."""
    H, T, last = 8, LONG, 200
    q, k, v, _ = inputs(1, H, 4, T, T, d, BF16, seed=311)
    lam = torch.where(torch.arange(H) % 2 == 0, 0.5, -0.5)
    ref, bound, _ = oa.diff(np64(q[:, :4, -last:]), np64(k[:, :2]), np64(v[:, :2]), np64(lam[:2]), NW, 0, d ** -0.5,
                            BITS[BF16], 8)
    v[0, 1, 5, 7] = float("inf")  # the second half of the first two pairs' values
    on = [t.to(dev) for t in (q, k, v, lam)]
    o, seconds = _seconds(lambda: lr.lr_fwd_diff(*on, norm=norm, eps=EPS, o=torch.full_like(on[0], 7.0)))
    assert lr.device_status() == LR_OK
    assert seconds < 1.0
    assert not (o[0, :, 5:] == 7).all(-1).any()
    assert o[0, 4:].isfinite().all() and o[0, :4, :5].isfinite().all()
    if norm:
        assert o[0, :2, 5:].isnan().all() and o[0, 3, 5:, 7].isnan().all()
        assert (o[0, 2, 5:] == 0).all() and (o[0, 3, 5:, :7] == 0).all() and (o[0, 3, 5:, 8:] == 0).all()
        return
    assert o[0, 1, 5:, 7].isnan().all() and (o[0, 3, 5:, 7] == float("inf")).all()
    got = o[:, :4, -last:].clone()
    got[:, 1::2, :, 7] = torch.from_numpy(ref[:, 1::2, :, 7]).to(dev)
    bound[:, 1::2, :, 7] += 1.0
    # rows that are computed again are rounded another way
    within(got, ref, 2 * bound)


@widths
def test_diff_squares_past_the_range_stay_quick(dev, d):
    """Finite values whose squares overflow: rows of zeros with the norm, without a
    second computation of every row; without it they are as they are."""
    T = LONG
    q, k, v, lam = inputs(1, 8, 8, T, T, d, BF16, seed=321)
    v.fill_(2.0 ** 70)
    on = [t.to(dev) for t in (q, k, v, lam)]
    usual = _seconds(lambda: lr.lr_fwd_diff(*[t.to(dev) for t in inputs(1, 8, 8, T, T, d, BF16, seed=321)]))[1]
    o, seconds = _seconds(lambda: lr.lr_fwd_diff(*on, eps=EPS))
    assert (o == 0).all()
    assert seconds < usual + 0.02
    o = np64(lr.lr_fwd_diff(*on, norm=False)) / 2.0 ** 70
    want = 1 - np.repeat(np64(lam), 2)[None, :, None, None]
    # the two means are off by the weights' rounding, 2^-8 each, and the result's
    assert (np.abs(o - want) <= 2.0 ** -7 * 2).all()


@types
@widths
def test_diff_rows_put_right_in_pieces_in_turn(dev, d, dtype):
    """More pieces than run at once, ragged, with NaN and infinities in some of them: the
    rows that see them, and no others."""
    B, H, T = 3, 16, 700
    q, k, v, lam = inputs(B, H, 4, T, T, d, dtype, seed=331)
    lens = [700, 389, 130]
    ref, bound, written = oa.diff(np64(q), np64(k), np64(v), np64(lam), 300, 2, d ** -0.5, BITS[dtype],
                                  8 if dtype == BF16 else None, None, None, lens, lens)
    nan, inf = float("nan"), float("inf")
    v[0, 0, 600, 1], v[1, 3, 50, 2], v[1, 3, 60, 2], v[2, 7, 129, d - 1] = nan, inf, -inf, nan
    ints = torch.tensor(lens, dtype=torch.int32, device=dev)
    o = torch.full(q.shape, 7.0, dtype=dtype, device=dev)
    lr.lr_fwd_diff(*(t.to(dev) for t in (q, k, v, lam)), window=300, sinks=2, norm=False, q_len=ints, k_len=ints, o=o)
    got, rows = np64(o), np.arange(T)
    for b, head, ch, sees in ((0, 0, 1, (rows >= 600)), (1, 1, 2, (rows >= 50) & (rows < 360)),
                              (2, 1, d - 1, rows >= 129)):
        pairs = {0: 0, 3: 1, 7: 3}[{0: 0, 1: 3, 2: 7}[b]]
        for h in range(4 * pairs, 4 * pairs + 4):
            at = sees & (rows < lens[b])
            assert np.isnan(got[b, 2 * h + head, at, ch]).all()
            got[b, 2 * h + head, at, ch] = ref[b, 2 * h + head, at, ch]
    w = np.broadcast_to(written[:, None, :, None], ref.shape)
    within(torch.from_numpy(got), np.where(w, ref, 7.0), np.where(w, 2 * bound, 0.0))


@types
@widths
@pytest.mark.parametrize("max_len", [65536, 131072])
def test_diff_step_beside_an_early_infinity(dev, max_len, d, dtype):
    """One sequence of 65536 tokens whose fourth holds an infinity: its channel, and the
    others as without it."""
    L, page = 65536, 256
    q = rnd(341, 1, 4, d, dtype=dtype)
    kc, vc = (rnd(342 + i, L // page, 2, page, d, dtype=dtype) for i in range(2))
    lam = torch.tensor([0.5, -0.5])
    table = torch.zeros(1, max_len // page, dtype=torch.int32)
    table[0, :L // page] = torch.arange(L // page)
    ref, bound, _ = oa.diff_step(np64(q), np64(kc), np64(vc), table.numpy(), [L], np64(lam), NW, 0, d ** -0.5,
                                 BITS[dtype], 8 if dtype == BF16 else None)
    vc[0, 1, 3, 2] = float("inf")
    on = [t.to(dev) for t in (q, kc, vc, table, torch.tensor([L], dtype=torch.int32), lam)]
    o, seconds = _seconds(lambda: lr.lr_step_paged_diff(*on, max_len=max_len, norm=False))
    assert seconds < 0.5
    assert o[0, 1, 2].isnan() and o[0, 3, 2] == float("inf")
    got = np64(o)
    got[0, 1::2, 2] = ref[0, 1::2, 2]
    within(torch.from_numpy(got), ref, 2 * bound)
    normed = lr.lr_step_paged_diff(*on, max_len=max_len)
    assert normed[0, :2].isnan().all() and normed[0, 3, 2].isnan() and (normed[0, 2] == 0).all()


@types
@widths
@pytest.mark.parametrize("top", [-58, -66, -73, -75, -110])
def test_diff_squares_below_the_range(dev, top, d, dtype):
    """Rows of one tiny channel, eps 0: their norm as long as the mean square is there
    (of 2^-140 it has nine bits), else times 2^74.5, and never an infinity."""
    q, k, v, _ = inputs(1, 2, 1, 5, 9, d, dtype, seed=351)
    v.zero_()
    v[0, 1, :, 4] = 2.0 ** top
    lam = torch.zeros(2, device=dev)
    args = [t.to(dev) for t in (q, k, v)]
    table = torch.zeros(1, 1, dtype=torch.int32, device=dev)
    pool = [torch.zeros(1, 2, 16, d, dtype=dtype, device=dev) for _ in range(2)]
    for p, t in zip(pool, args[1:]):
        p[0, :, :9] = t[0]
    rows = lr.lr_fwd_diff(*args, lam, eps=0.0)[0, :, -1]
    step = lr.lr_step_paged_diff(args[0][:, :, -1].contiguous(), *pool, table,
                                 torch.tensor([9], dtype=torch.int32, device=dev), lam, eps=0.0)[0]
    # 2 d channels of which one is not zero: sqrt(2 d)
    x = (2 * d) ** 0.5 if top >= -66 else 2.0 ** (top + 74.5)
    # the weights are off by up to 2^-8 each in bf16, the result by as much; the mean by 2^-10
    for o in (rows, step):
        o = np64(o)
        assert (np.abs(o[1::2, 4] - x) <= x * (3 * 2.0 ** -8 if dtype == BF16 else 2.0 ** -10)).all()
        o[1::2, 4] = 0
        assert (o == 0).all()


@widths
def test_diff_weights_count_the_same_anywhere_in_a_tile(dev, d):
    """A row on two keys, one in each of two tiles of 128: the same bits for every place
    of either, and right."""
    B, T = 128, 256
    q, k = torch.zeros(B, 2, 1, d), torch.zeros(B, 2, T, d)
    q[:, 0, :, 0], q[:, 1, :, 0] = 1.0, 1.25
    k[..., 0] = -1000.0
    v = rnd(361, 1, 2, 2, d, dtype=BF16)
    values = rnd(362, B, 2, T, d, dtype=BF16)
    for b in range(B):
        first, second = b, 128 + (37 * b + 11) % 128
        k[b, :, first, 0], k[b, :, second, 0] = 0.0, -1.203125
        values[b, :, first], values[b, :, second] = v[0, :, 0], v[0, :, 1]
    lam = torch.tensor([0.5])
    o = lr.lr_fwd_diff(*(t.to(BF16).to(dev) for t in (q, k, values)), lam.to(dev), scale=1.0, norm=False)
    ref, bound, _ = oa.diff(np64(q[:1]), np64(k[:1]), np64(values[:1]), np64(lam), NW, 0, 1.0, BITS[BF16], 8)
    within(o, np.broadcast_to(ref, o.shape), np.broadcast_to(bound, o.shape))
    assert torch.equal(o, o[:1].expand_as(o))


@types
@widths
def test_diff_equal_maps_cancel(dev, d, dtype):
    """The same map twice and lambda 1, over several tiles and pieces: zeros, whatever eps."""
    q, k, v, _ = inputs(2, 3, 1, 300, 700, d, dtype, seed=371)
    q[:, 1::2], k[:, 1::2] = q[:, 0::2], k[:, 0::2]
    one = torch.ones(3, device=dev)
    for norm, eps, window in ((False, 0.0, None), (True, 0.0, 90), (True, EPS, None)):
        o = lr.lr_fwd_diff(*(t.to(dev) for t in (q, k, v)), one, norm=norm, eps=eps, window=window, sinks=3)
        assert (o == 0).all()


@types
@widths
@pytest.mark.parametrize("scale", [1.0, -1.0])
@pytest.mark.parametrize("top", [2.0 ** 33, 2.0 ** 66, 2.0 ** 126], ids=str)
def test_diff_scores_far_above_the_others(dev, top, scale, d, dtype):
    """Scores of 1e10 and more, one a 64th part above the others in each map, in the
    first and in the last tile: each map gives its value alone."""
    Tq, Tk = 30, 300
    q, k, v, lam = inputs(1, 1, 1, Tq, Tk, d, dtype, seed=381)
    q.zero_(), k.zero_()
    q[..., 0] = scale
    k[..., 0] = torch.tensor(top * (1 - 2.0 ** -6))
    k[0, 0, 250, 0] = k[0, 1, 17, 0] = top
    o = lr.lr_fwd_diff(*(t.to(dev) for t in (q, k, v)), lam.to(dev), scale=scale, norm=False)
    row = torch.cat((v[0, 0], v[0, 1]), -1).double()
    want = (row[250] - float(lam[0]) * row[17]).view(2, 1, d).expand(2, Tq, d)
    within(o[0], np64(want), np.abs(np64(want)) * 2.0 ** -BITS[dtype] + 2.0 ** -22)


@types
@widths
def test_diff_weights_keep_sixteen_bits(dev, d, dtype):
    """Maps that differ little and lambda 1, rows on few keys: what is left of the values
    is small beside the weights' rounding to 8 bits, so only wider ones come within the bound."""
    T = 150
    q, k, v, _ = inputs(1, 2, 2, T, T, d, dtype, seed=391)
    q[:, 1::2] = q[:, 0::2]
    k[:, 1::2] = (k[:, 0::2].float() + 0.02 * rnd(392, 1, 2, T, d)).to(dtype)
    lam = torch.ones(2)
    ref, bound, _ = oa.diff(np64(q), np64(k), np64(v), np64(lam), 40, 2, d ** -0.5, BITS[dtype],
                            16 if dtype == BF16 else None)
    o = lr.lr_fwd_diff(*(t.to(dev) for t in (q, k, v, lam)), window=40, sinks=2, norm=False)
    within(o, ref, bound)
    # the step of the last token, its cache in pages of 16
    pages = -(-T // 16)
    pool = [torch.zeros(pages * 16, 4, d, dtype=dtype, device=dev) for _ in range(2)]
    for p, t in zip(pool, (k, v)):
        p[:T] = t[0].transpose(0, 1)
    pool = [p.view(pages, 16, 4, d).transpose(1, 2).contiguous() for p in pool]
    o = lr.lr_step_paged_diff(q[:, :, -1].contiguous().to(dev), *pool,
                              torch.arange(pages, dtype=torch.int32, device=dev)[None],
                              torch.tensor([T], dtype=torch.int32, device=dev), lam.to(dev), window=40, sinks=2,
                              norm=False)
    within(o, ref[:, :, -1], bound[:, :, -1])
