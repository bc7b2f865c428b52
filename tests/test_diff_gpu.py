"""lr_fwd_diff against its fp64 definition (oracle/attention.py), element by
element within the bound derived there, at the sizes, masks, strides and
lengths where a kernel can go wrong.
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


def check(dev, q, k, v, lam, window, sinks, scale=None, q_len=None, k_len=None, norm=True, weight=None, views=None,
          what=""):
    dtype, d = q.dtype, q.shape[-1]
    scale = d ** -0.5 if scale is None else scale
    lay = views or (lambda t: t)
    o = lay(torch.full(q.shape, 7.0, dtype=dtype, device=dev))
    ints = [None if x is None else torch.tensor(x, dtype=torch.int32, device=dev) for x in (q_len, k_len)]
    out = lr.lr_fwd_diff(*(lay(t.to(dev)) for t in (q, k, v)), lam.to(dev), window=window, sinks=sinks,
                         q_len=ints[0], k_len=ints[1], scale=scale, norm=norm, eps=EPS,
                         norm_weight=None if weight is None else weight.to(dev), o=o)
    torch.cuda.synchronize()
    assert out is o
    ref, bound, written = oa.diff(np64(q), np64(k), np64(v), np64(lam), window, sinks, scale, BITS[dtype],
                                  8 if dtype == BF16 else None, None if weight is None else np64(weight),
                                  EPS if norm else None, q_len, k_len)
    w = np.broadcast_to(written[:, None, :, None], ref.shape)
    within(out, np.where(w, ref, 7.0), np.where(w, bound, 0.0), what)
    return out


SHAPES = [  # B, H, Hk, Tq, Tk, window, sinks
    (1, 1, 1, 1, 1, NW, 0), (1, 2, 1, 1, 5, 3, 1), (2, 3, 3, 7, 7, 1, 0), (1, 4, 2, 63, 63, 16, 4),
    (2, 4, 1, 65, 65, 64, 0), (1, 2, 1, 128, 128, 128, 0), (1, 3, 1, 129, 129, 63, 65), (1, 2, 2, 200, 333, 100, 4),
    (1, 8, 1, 33, 400, 50, 70), (1, 2, 1, 257, 257, NW, 0), (1, 5, 5, 130, 400, 129, 1), (1, 2, 2, 2, 260, 1, 5),
    (3, 2, 1, 40, 300, 300, 0), (1, 1, 1, 300, 1100, NW, 0),
]


@types
@pytest.mark.parametrize("norm", [True, False], ids=["norm", "plain"])
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join("inf" if x == NW else str(x) for x in s))
def test_diff_parity(dev, shape, d, norm, dtype):
    B, H, Hk, Tq, Tk, window, sinks = shape
    q, k, v, lam = inputs(B, H, Hk, Tq, Tk, d, dtype)
    check(dev, q, k, v, lam, window, sinks, norm=norm, weight=rnd(9, 2 * d) if norm and H > 1 else None)


@types
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("window,sinks", [(NW, 0), (200, 4)])
def test_diff_more_pieces_than_run_at_once(dev, window, sinks, d, dtype):
    """Every CTA takes several pieces, of all lengths, some without rows."""
    B, H, T = 3, 16, 1000
    q, k, v, lam = inputs(B, H, 4, T, T, d, dtype, seed=11)
    check(dev, q, k, v, lam, window, sinks, q_len=[1000, 130, 0], k_len=[1000, 700, 40], weight=rnd(14, 2 * d))


@types
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (7, 0), (130, 3), (33, 50), (NW, 4)])
def test_diff_sees_each_key_once(dev, window, sinks, d, dtype):
    """Zero keys, so that every seen key has the same weight in both maps, and
    values that mark the key: the output is (1 - lambda) / n for every key seen."""
    T, H = 300, 2
    q, k, v, lam = inputs(1, H, 1, T, T, d, dtype, seed=21)
    k.zero_()
    v.zero_()
    for j in range(T):
        v[0, (j // d) % 2, j, j % d] = 1
    check(dev, q, k, v, lam, window, sinks, norm=False)


@types
@pytest.mark.parametrize("d", [64, 128])
def test_diff_of_one_map_is_the_window(dev, d, dtype):
    """lambda 0: the first map's attention over both halves of the values."""
    q, k, v, _ = inputs(2, 3, 3, 150, 260, d, dtype, seed=31)
    qd, kd, vd = (t.to(dev) for t in (q, k, v))
    o = lr.lr_fwd_diff(qd, kd, vd, torch.zeros(3, device=dev), window=70, sinks=3, norm=False)
    for half in range(2):
        ref, size, reach, _ = oa.window(np64(q[:, 0::2]), np64(k[:, 0::2]), np64(v[:, half::2]), 70, 3, d ** -0.5)
        bound = oa.attention_bound(ref, size, reach, 260, d, BITS[dtype], 8 if dtype == BF16 else None)
        within(o[:, half::2], ref, bound)
        a = lr.lr_fwd_window(qd[:, 0::2], kd[:, 0::2], vd[:, half::2], window=70, sinks=3)
        within(o[:, half::2], np64(a), 2 * bound)


@types
def test_diff_maps_that_cancel_give_zeros(dev, dtype):
    """The same map twice and lambda 1: zeros, with the norm too, whatever eps."""
    q, k, v, _ = inputs(1, 2, 1, 70, 200, 64, dtype, seed=36)
    q[:, 1::2], k[:, 1::2] = q[:, 0::2], k[:, 0::2]
    one = torch.ones(2, device=dev)
    for norm, eps in ((False, 0.0), (True, 0.0), (True, EPS)):
        o = lr.lr_fwd_diff(*(t.to(dev) for t in (q, k, v)), one, norm=norm, eps=eps)
        assert (o == 0).all()


@types
@pytest.mark.parametrize("d", [32, 64, 128])
def test_diff_ragged_batch_with_garbage_in_the_padding(dev, d, dtype):
    """Lengths from none on, rows before the first key, NaN and infinities
    behind every sequence."""
    B, Tq, Tk = 5, 150, 400
    q_len, k_len = [150, 7, 0, 33, 140], [400, 3, 200, 0, 129]
    q, k, v, lam = inputs(B, 2, 1, Tq, Tk, d, dtype, seed=41)
    ref, bound, written = oa.diff(np64(q), np64(k), np64(v), np64(lam), 90, 4, d ** -0.5, BITS[dtype],
                                  8 if dtype == BF16 else None, None, EPS, q_len, k_len)
    for b in range(B):
        q[b, :, q_len[b]:] = float("nan")
        k[b, :, k_len[b]:] = float("nan")
        v[b, :, k_len[b]:] = float("inf")
    o = torch.full(q.shape, 7.0, dtype=dtype, device=dev)
    ql, kl = (torch.tensor(x, dtype=torch.int32, device=dev) for x in (q_len, k_len))
    lr.lr_fwd_diff(*(t.to(dev) for t in (q, k, v)), lam.to(dev), window=90, sinks=4, q_len=ql, k_len=kl, eps=EPS, o=o)
    w = np.broadcast_to(written[:, None, :, None], ref.shape)
    within(o, np.where(w, ref, 7.0), np.where(w, bound, 0.0))
    made = lr.lr_fwd_diff(*(t.to(dev) for t in (q, k, v)), lam.to(dev), window=90, sinks=4, q_len=ql, k_len=kl, eps=EPS)
    assert torch.equal(made, torch.where(torch.from_numpy(w.copy()).to(dev), o, torch.zeros_like(o)))


@types
@pytest.mark.parametrize("norm", [True, False], ids=["norm", "plain"])
@pytest.mark.parametrize("d", [32, 64, 128])
def test_diff_masked_values_cannot_reach_other_rows(dev, d, norm, dtype):
    """Keys in the middle are NaN and infinite: rows that do not see them are as without them."""
    T = 300
    q, k, v, lam = inputs(1, 2, 2, T, T, d, dtype, seed=51)
    args = dict(window=40, sinks=2, norm=norm)
    want = lr.lr_fwd_diff(*(t.to(dev) for t in (q, k, v)), lam.to(dev), **args).cpu()
    _, bound, _ = oa.diff(np64(q), np64(k), np64(v), np64(lam), 40, 2, d ** -0.5, BITS[dtype],
                          8 if dtype == BF16 else None, None, EPS if norm else None)
    k[0, 1, 100] = float("nan")
    v[0, 0, 101, 3], v[0, 3, 102, 5] = float("inf"), float("nan")
    got = lr.lr_fwd_diff(*(t.to(dev) for t in (q, k, v)), lam.to(dev), **args).cpu()
    rows = np.arange(T)
    for h, at in ((0, (100, 101)), (1, (102,))):
        sees = np.zeros(T, bool)
        for j in at:
            sees |= (rows >= j) & (rows < j + 40)
        heads = slice(2 * h, 2 * h + 2)
        # rows beside them may be computed another way, within the bound
        within(got[:, heads, ~sees], np64(want[:, heads, ~sees]), 2 * bound[:, heads][:, :, ~sees])
        far = ~sees & (rows > 270)
        assert torch.equal(got[:, heads, far], want[:, heads, far])


@types
@pytest.mark.parametrize("d", [32, 64, 128])
def test_diff_seen_infinities_and_nan(dev, d, dtype):
    """Without the norm a channel is the difference of the maps' channels: a seen
    infinity is one in both, so NaN where lambda is positive and that infinity where
    it is negative; a NaN stays in its channel; a NaN key makes the pair NaN.  With
    the norm the mean square is infinite or NaN: other channels 0 or NaN."""
    T, inf, nan = 40, float("inf"), float("nan")
    q, k, v, _ = inputs(3, 2, 1, 4, T, d, dtype, seed=61)
    lam = torch.tensor([0.5, -0.5])
    ref, bound, _ = oa.diff(np64(q), np64(k), np64(v), np64(lam), NW, 0, d ** -0.5, BITS[dtype],
                            8 if dtype == BF16 else None)
    v[0, 0, 9, 3], v[0, 1, 11, 4], v[1, 1, 9, 6], k[2, 1, 9, 1] = inf, -inf, nan, nan
    run = lambda norm: lr.lr_fwd_diff(*(x.to(dev) for x in (q, k, v)), lam.to(dev), norm=norm, eps=EPS).cpu()
    got = run(False)
    for b, head, ch, x in ((0, 0, 3, nan), (0, 2, 3, inf), (0, 1, 4, nan), (0, 3, 4, -inf), (1, 1, 6, nan), (1, 3, 6, nan)):
        assert np.array_equal(np64(got[b, head, :, ch]), np.full(4, x), equal_nan=True), (b, head)
        got[b, head, :, ch] = 0
        ref[b, head, :, ch] = 0
    within(got[:2], ref[:2], 2 * bound[:2])
    assert got[2].isnan().all()
    normed = run(True)
    assert normed[0, :2].isnan().all() and normed[1].isnan().all() and normed[2].isnan().all()
    assert normed[0, 2, :, 3].isnan().all() and normed[0, 3, :, 4].isnan().all()
    normed[0, 2, :, 3] = normed[0, 3, :, 4] = 0
    assert (normed[0, 2:] == 0).all()


@types
@pytest.mark.parametrize("d", [32, 64, 128])
def test_diff_seen_infinities_in_one_tile_of_many_pieces(dev, d, dtype):
    """As above with keys that no CTAs share out, in every batch and pair: each half of
    a row is put right by itself, and rows before the infinity do not know of it."""
    B, H, T, inf = 20, 8, 30, float("inf")
    q, k, v, lam = inputs(B, H, 4, T, T, d, dtype, seed=65)
    ref, bound, _ = oa.diff(np64(q), np64(k), np64(v), np64(lam), NW, 0, d ** -0.5, BITS[dtype],
                            8 if dtype == BF16 else None)
    v[:, 1, 9, d - 1] = inf  # the second half of the first pair's values, a positive lambda
    got = np64(lr.lr_fwd_diff(*(x.to(dev) for x in (q, k, v)), lam.to(dev), norm=False))
    assert np.isnan(got[:, 1:4:2, 9:, d - 1]).all()
    got[:, 1:4:2, 9:, d - 1] = ref[:, 1:4:2, 9:, d - 1]
    # rows that are computed again are rounded another way
    within(torch.from_numpy(got), ref, 2 * bound)
    normed = np64(lr.lr_fwd_diff(*(x.to(dev) for x in (q, k, v)), lam.to(dev), eps=EPS))
    assert np.isnan(normed[:, :4, 9:]).all() and np.isfinite(normed[:, :4, :9]).all() and np.isfinite(normed[:, 4:]).all()


@types
@pytest.mark.parametrize("d", [32, 64, 128])
def test_diff_calls_in_a_row_on_one_workspace(dev, d, dtype):
    B, H, T, tries = 2, 3, 400, 6
    sets = [inputs(B, H, 1, T, T, d, dtype, seed=200 + 10 * i) for i in range(tries)]
    sets = [[t.to(dev) for t in x] for x in sets]
    size = lr.diff_workspace_size(B, H, 1, T, T, d, dtype)
    ws = torch.empty(max(size, 1), dtype=torch.uint8, device=dev)
    want = []
    for q, k, v, lam in sets:
        want.append(lr.lr_fwd_diff(q, k, v, lam, window=150, workspace=ws))
        torch.cuda.synchronize()
        ws.fill_(255)
    now, got = [t.clone() for t in sets[0]], []
    for x in sets:
        for a, b in zip(now, x):
            a.copy_(b)
        got.append(lr.lr_fwd_diff(*now, window=150, workspace=ws))
        ws.fill_(255)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@types
@pytest.mark.parametrize("which", ["k", "v"])
def test_diff_batch_full_of_nan_stays_quick(dev, which, dtype):
    import time
    q, k, v, lam = inputs(1, 8, 8, 2048, 2048, 64, dtype, seed=71)
    (k if which == "k" else v).fill_(float("nan"))
    qd, kd, vd, ld = (t.to(dev) for t in (q, k, v, lam))
    lr.lr_fwd_diff(qd, kd, vd, ld)
    torch.cuda.synchronize()
    t0 = time.time()
    o = lr.lr_fwd_diff(qd, kd, vd, ld)
    torch.cuda.synchronize()
    assert time.time() - t0 < 1.0
    assert o.isnan().all()


@types
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("scale", [0.0, -0.3, 1e-3, 2.0])
def test_diff_scales(dev, scale, d, dtype):
    q, k, v, lam = inputs(1, 2, 1, 60, 190, d, dtype, seed=81)
    lam[1] = -0.7
    check(dev, q, k, v, lam, 100, 3, scale=scale, norm=scale != 0.0)


@types
@pytest.mark.parametrize("top", [2.0 ** 33, 2.0 ** 66, 2.0 ** 126], ids=str)
def test_diff_large_finite_scores(dev, top, dtype):
    """Scores of 1e10 and more, one a 64th part above the others in each map:
    each map gives its value alone."""
    d, Tq, Tk = 64, 30, 300
    q, k, v, lam = inputs(1, 1, 1, Tq, Tk, d, dtype, seed=91)
    q.zero_(), k.zero_()
    q[..., 0] = 1
    k[..., 0] = torch.tensor(top * (1 - 2.0 ** -6))
    k[0, 0, 250, 0] = k[0, 1, 17, 0] = top
    o = lr.lr_fwd_diff(*(t.to(dev) for t in (q, k, v)), lam.to(dev), scale=1.0, norm=False)
    row = torch.cat((v[0, 0], v[0, 1]), -1).double()
    want = (row[250] - float(lam[0]) * row[17]).view(2, 1, d).expand(2, Tq, d)
    within(o[0], np64(want), np.abs(np64(want)) * 2.0 ** -BITS[dtype] + 2.0 ** -22)


@types
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("part", [1.0, 0.5])
def test_diff_values_at_the_end_of_the_type(dev, part, d, dtype):
    """Means of the type's largest values do not overflow; with the norm their
    squares do, and the row is divided by infinity."""
    T = 260
    q, k, v, _ = inputs(1, 2, 1, T, T, d, dtype, seed=95)
    v.fill_(torch.finfo(dtype).max * part)
    lam = torch.tensor([0.5, 0.25], device=dev)
    o = np64(lr.lr_fwd_diff(*(t.to(dev) for t in (q, k, v)), lam, norm=False))
    top = float(v.double()[0, 0, 0, 0])
    for h, x in enumerate((0.5, 0.75)):
        # the two means are off by the weights' rounding, 2^-8 each in bf16
        assert (np.abs(o[0, 2 * h:2 * h + 2] / top - x) <= (2.0 ** -7 if dtype == BF16 else 2.0 ** -14)).all()
    assert (lr.lr_fwd_diff(*(t.to(dev) for t in (q, k, v)), lam) == 0).all()


def _tokens_first(t):
    return t.transpose(1, 2).contiguous().transpose(1, 2)


def _padded(t):
    big = torch.full((*t.shape[:2], t.shape[2] + 3, t.shape[3] + 32), 5.0, dtype=t.dtype, device=t.device)
    view = big[:, :, 1:-2, 16:-16]
    view.copy_(t)
    return view


@types
@pytest.mark.parametrize("views", [_tokens_first, _padded], ids=["tokens-first", "padded"])
@pytest.mark.parametrize("d", [32, 64, 128])
def test_diff_strided_tensors(dev, d, views, dtype):
    q, k, v, lam = inputs(2, 4, 2, 140, 270, d, dtype, seed=101)
    check(dev, q, k, v, lam, 150, 4, q_len=[140, 61], k_len=[270, 200], views=views)


@types
def test_diff_offsets_past_32_bits(dev, dtype):
    """Strides that carry the last head past 2^31 elements."""
    d, T = 64, 200
    q, k, v, lam = inputs(1, 1, 1, T, T, d, dtype, seed=111)
    want = lr.lr_fwd_diff(*(t.to(dev) for t in (q, k, v)), lam.to(dev))
    far = []
    for t in (q, k, v, torch.zeros_like(q)):
        room = torch.empty((1 << 31) + T * d + 64, dtype=dtype, device=dev)
        view = torch.as_strided(room, (1, 2, T, d), (d, 1 << 31, d, 1))
        view.copy_(t)
        far.append(view)
    got = lr.lr_fwd_diff(*far[:3], lam.to(dev), o=far[3])
    assert torch.equal(got, want)


def test_diff_lengths_out_of_range_are_reported(dev):
    for dtype in (F32, BF16):
        q, k, v, lam = (t.to(dev) for t in inputs(2, 1, 1, 20, 30, 64, dtype, seed=121))
        good = lr.lr_fwd_diff(q, k, v, lam)
        assert lr.device_status() == LR_OK
        for ql, kl in (([21, 20], [30, 30]), ([20, 20], [30, 31]), ([2 ** 31 - 1, 20], [30, 30])):
            o = lr.lr_fwd_diff(q, k, v, lam, q_len=torch.tensor(ql, dtype=torch.int32, device=dev),
                               k_len=torch.tensor(kl, dtype=torch.int32, device=dev))
            assert lr.device_status() == LR_ERR_INDEX and lr.device_status() == LR_OK
            assert torch.equal(o, good)


@types
def test_diff_empty_calls(dev, dtype):
    q, k, v, lam = (t.to(dev) for t in inputs(2, 1, 1, 5, 4, 64, dtype, seed=131))
    assert lr.lr_fwd_diff(q[:, :, :0], k, v, lam).shape == (2, 2, 0, 64)
    assert (lr.lr_fwd_diff(q, k[:, :, :0], v[:, :, :0], lam) == 0).all()
    o = torch.full_like(q, 7.0)
    lr.lr_fwd_diff(q, k[:, :, :0], v[:, :, :0], lam, q_len=torch.tensor([2, 0], dtype=torch.int32, device=dev), o=o)
    assert (o[0, :, :2] == 0).all() and (o[0, :, 2:] == 7).all() and (o[1] == 7).all()


@types
def test_diff_captures_into_graphs_that_share_a_workspace(dev, dtype):
    """Replays follow inputs, lengths and lambda; two graphs use one workspace in turn."""
    B, H, T, d = 3, 4, 500, 64
    q, k, v, lam = (t.to(dev) for t in inputs(B, H, H, T, T, d, dtype, seed=141))
    ql = torch.tensor([500, 300, 5], dtype=torch.int32, device=dev)
    need = lr.diff_workspace_size(B, H, H, T, T, d, dtype)
    assert (need > 0) == (dtype == F32)
    ws = torch.empty(max(need, 16), dtype=torch.uint8, device=dev)
    call = lambda window: lr.lr_fwd_diff(q, k, v, lam, window=window, q_len=ql, k_len=ql, workspace=ws)
    call(None), call(100)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for window in (None, 100):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(call(window))
        graphs.append(g)
    for s in range(3):
        q.copy_(rnd(145 + s, *q.shape, dtype=dtype))
        lam.mul_(0.9)
        for i, window in ((0, None), (1, 100), (0, None)):
            graphs[i].replay()
            assert torch.equal(outs[i], call(window))
        ql -= 2


@types
def test_diff_two_calls_at_once_and_another_stream(dev, dtype):
    q, k, v, lam = (t.to(dev) for t in inputs(2, 4, 2, 1500, 1500, 128, dtype, seed=151))
    want = [lr.lr_fwd_diff(q, k, v, lam, window=w) for w in (None, 300)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(dev) for _ in range(2)]
    for _ in range(3):
        got = []
        for s, w in zip(streams, (None, 300)):
            got.append(lr.lr_fwd_diff(q, k, v, lam, window=w, stream=s))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
