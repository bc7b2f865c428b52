"""Parity of the attention entry points (lr_qk_norm_rope, lr_fwd_window,
lr_step_paged) with their fp64 definition (oracle/attention.py), element by
element within ``attention_bound``'s derived bounds, at the sizes, masks,
strides and lengths where a kernel can go wrong.
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


def check_window(dev, q, k, v, window, sinks, scale, q_len=None, k_len=None, dtype=F32, views=None, what=""):
    """Runs the call on device copies (laid out by `views`), compares rows
    that are written with the oracle and the others with their old content."""
    d = q.shape[-1]
    qd, kd, vd = (t.to(dev) for t in (q, k, v))
    if views:
        qd, kd, vd = views(qd), views(kd), views(vd)
    o = torch.full(q.shape, 7.0, dtype=dtype, device=dev)
    if views:
        o = views(o)
    ints = [None if x is None else torch.tensor(x, dtype=torch.int32, device=dev) for x in (q_len, k_len)]
    out = lr.lr_fwd_window(qd, kd, vd, window=window, sinks=sinks, q_len=ints[0], k_len=ints[1], scale=scale, o=o)
    torch.cuda.synchronize()
    assert out is o
    ref, size, reach, written = oa.window(np64(q), np64(k), np64(v), window, sinks, scale, q_len, k_len)
    bound = oa.attention_bound(ref, size, reach, k.shape[2], d, BITS[dtype], 8 if dtype == BF16 else None)
    w = np.broadcast_to(written[:, None, :, None], ref.shape)
    within(out, np.where(w, ref, 7.0), np.where(w, bound, 0.0), what)


SHAPES = [  # B, Hq, Hk, Tq, Tk, window, sinks
    (1, 1, 1, 1, 1, NW, 0), (1, 2, 1, 1, 5, 3, 1), (2, 3, 3, 7, 7, 1, 0), (1, 4, 2, 63, 63, 16, 4),
    (1, 2, 2, 64, 64, NW, 0), (2, 4, 1, 65, 65, 64, 0), (1, 6, 2, 127, 127, 32, 3), (1, 2, 1, 128, 128, 128, 0),
    (1, 3, 1, 129, 129, 63, 65), (1, 2, 2, 200, 333, 100, 4), (1, 8, 1, 33, 400, 50, 70), (1, 2, 1, 257, 257, NW, 0),
    (1, 5, 5, 130, 400, 129, 1), (1, 4, 4, 300, 300, 65, 130), (1, 2, 2, 2, 260, 1, 5), (3, 2, 1, 40, 300, 300, 0),
]


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join("inf" if x == NW else str(x) for x in s))
def test_window_parity(dev, shape, d, dtype):
    B, Hq, Hk, Tq, Tk, window, sinks = shape
    q, k, v = (rnd(s, B, h, t, d, dtype=dtype) for s, h, t in ((1, Hq, Tq), (2, Hk, Tk), (3, Hk, Tk)))
    check_window(dev, q, k, v, window, sinks, d ** -0.5, dtype=dtype)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("d,Hq,Hk", [(32, 1, 1), (64, 2, 1), (128, 3, 1), (128, 4, 2)])
@pytest.mark.parametrize("Tq,Tk,window,sinks", [(1, 700, NW, 0), (3, 1100, 600, 4), (130, 900, NW, 0), (129, 1500, 1200, 200),
                                                (300, 520, NW, 3), (17, 4000, NW, 0)])
def test_window_few_rows_and_many_keys(dev, dtype, d, Hq, Hk, Tq, Tk, window, sinks):
    """Few pieces of work: the keys are shared out over the CTAs of a cluster."""
    q, k, v = (rnd(s, 1, h, t, d, dtype=dtype) for s, h, t in ((100, Hq, Tq), (101, Hk, Tk), (102, Hk, Tk)))
    check_window(dev, q, k, v, window, sinks, d ** -0.5, dtype=dtype)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_window_few_rows_ragged_empty_and_not_finite(dev, dtype):
    """The same with lengths from none on, NaN in the padding, parts of a
    cluster without any key, a NaN that some rows see and a masked infinity."""
    B, d, Tq, Tk = 4, 128, 40, 1400
    q_len, k_len = [40, 7, 0, 33], [1400, 3, 900, 0]
    q, k, v = (rnd(s, B, 2, t, d, dtype=dtype) for s, t in ((103, Tq), (104, Tk), (105, Tk)))
    ref, size, reach, written = oa.window(*(np64(t) for t in (q, k, v)), 1300, 2, d ** -0.5, q_len, k_len)
    bound = oa.attention_bound(ref, size, reach, Tk, d, BITS[dtype], 8 if dtype == BF16 else None)
    for b in range(B):
        k[b, :, k_len[b]:] = float("nan")
        v[b, :, k_len[b]:] = float("inf")
    v[0, 0, 70, 5] = float("inf")   # rows at 1360.. see keys from 61.. on, those at 1371.. not key 70
    o = torch.full(q.shape, 7.0, dtype=dtype, device=dev)
    ql, kl = (torch.tensor(x, dtype=torch.int32, device=dev) for x in (q_len, k_len))
    lr.lr_fwd_window(q.to(dev), k.to(dev), v.to(dev), window=1300, sinks=2, q_len=ql, k_len=kl, o=o)
    o = o.cpu()
    sees = [oa.sees(1360 + i, 70, 1400, 1300, 2) for i in range(Tq)]
    assert 0 < sum(sees) < Tq
    assert all((o[0, 0, i, 5] == float("inf")) == sees[i] for i in range(Tq))
    o[0, 0, torch.tensor(sees), 5] = 0
    ref[0, 0, sees, 5], bound[0, 0, sees, 5] = 0, 0
    w = np.broadcast_to(written[:, None, :, None], ref.shape)
    within(o, np.where(w, ref, 7.0), np.where(w, bound, 0.0))


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("d,Tq,Tk", [(32, 1, 1100), (128, 2, 300), (64, 65, 200)])
@pytest.mark.parametrize("H", [5, 13, 15, 16, 19, 23, 27, 33, 37, 45, 70, 76, 77, 150])
def test_window_cluster_sizes(dev, dtype, d, Tq, Tk, H):
    """Numbers of heads that are given to clusters of every size and to none,
    with fewer and more key tiles than CTAs."""
    q, k, v = (rnd(s, 1, H, t, d, dtype=dtype) for s, t in ((109, Tq), (110, Tk), (111, Tk)))
    check_window(dev, q, k, v, NW, 0, d ** -0.5, dtype=dtype)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_window_cluster_lengths(dev, dtype):
    """Shared pieces where the lengths leave a CTA many tiles, one, or none."""
    B, d, Tq, Tk = 6, 64, 70, 900
    q, k, v = (rnd(s, B, 2, t, d, dtype=dtype) for s, t in ((112, Tq), (113, Tk), (114, Tk)))
    for window, sinks in ((NW, 0), (300, 0), (300, 150)):
        check_window(dev, q, k, v, window, sinks, d ** -0.5, [70, 1, 69, 70, 0, 3], [900, 128, 33, 70, 500, 897],
                     dtype=dtype)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("Tk", [40, 1400])
def test_window_infinite_value_of_a_key_without_weight(dev, Tk, dtype):
    """A seen infinity shows even where the weight of its key, and of all keys
    that are worked on with it, rounds to zero."""
    d = 64
    q, k, v = (rnd(s, 1, 1, t, d, dtype=dtype) for s, t in ((106, 4), (107, Tk), (108, Tk)))
    q[..., 0] = 8
    k[..., 0] = 0
    k[:, :, :Tk // 2, 0] = -512     # scores 512 below the others'
    v[0, 0, 3, 9] = float("-inf")
    o = lr.lr_fwd_window(q.to(dev), k.to(dev), v.to(dev)).cpu()
    assert (o[0, 0, :, 9] == float("-inf")).all()
    o[..., 9] = 0
    v[0, 0, 3, 9] = 0
    ref, size, reach, _ = oa.window(*(np64(t) for t in (q, k, v)), NW, 0, d ** -0.5)
    bound = oa.attention_bound(ref, size, reach, Tk, d, BITS[dtype], 8 if dtype == BF16 else None)
    ref[..., 9], bound[..., 9] = 0, 0
    within(o, ref, bound)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("window,sinks", [(1, 0), (5, 2), (64, 0), (64, 64), (100, 130), (NW, 0)])
def test_window_sees_each_key_once(dev, window, sinks, dtype):
    """Zero keys weigh all seen keys alike; values that mark the key by its
    residue modulo d count the keys of each residue, so a key missed, doubled
    or shown in error changes a count by one: 1 / count of an output, over a
    hundred times a bf16 rounding of it at these lengths."""
    T, d = 290, 128
    q = rnd(4, 1, 2, T, d, dtype=dtype)
    k = torch.zeros(1, 1, T, d, dtype=dtype)
    v = torch.zeros(1, 1, T, d, dtype=dtype)
    v[0, 0, torch.arange(T), torch.arange(T) % d] = 1
    check_window(dev, q, k, v, window, sinks, 1.0, dtype=dtype)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("window,sinks", [(NW, 0), (40, 3)])
def test_window_ragged_batch_with_garbage_in_the_padding(dev, dtype, window, sinks):
    """Lengths from none to all; NaN and infinities behind every length; rows
    whose position is negative see nothing and are zeros; rows behind q_len
    keep their content."""
    B, Hq, Hk, Tq, Tk, d = 7, 4, 2, 150, 210, 64
    q_len, k_len = [150, 0, 1, 149, 60, 90, 17], [210, 5, 1, 180, 0, 70, 200]
    q, k, v = (rnd(s, B, h, t, d, dtype=dtype) for s, h, t in ((5, Hq, Tq), (6, Hk, Tk), (7, Hk, Tk)))
    clean = [t.clone() for t in (q, k, v)]
    for b in range(B):
        q[b, :, q_len[b]:] = float("nan")
        k[b, :, k_len[b]:] = float("nan")
        v[b, :, k_len[b]:] = float("inf") if b % 2 else float("nan")
    qd, kd, vd = (t.to(dev) for t in (q, k, v))
    o = torch.full(q.shape, 7.0, dtype=dtype, device=dev)
    ql, kl = (torch.tensor(x, dtype=torch.int32, device=dev) for x in (q_len, k_len))
    lr.lr_fwd_window(qd, kd, vd, window=window, sinks=sinks, q_len=ql, k_len=kl, o=o)
    torch.cuda.synchronize()
    ref, size, reach, written = oa.window(*(np64(t) for t in clean), window, sinks, d ** -0.5, q_len, k_len)
    bound = oa.attention_bound(ref, size, reach, Tk, d, BITS[dtype], 8 if dtype == BF16 else None)
    w = np.broadcast_to(written[:, None, :, None], ref.shape)
    within(o, np.where(w, ref, 7.0), np.where(w, bound, 0.0))


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_window_masked_values_cannot_reach_other_rows(dev, dtype, d, bad):
    """One non-finite key row and one non-finite value row: rows that see them
    become non-finite (or follow the formula), all others equal the result
    without them bit for bit or within the bound."""
    T, window, at = 300, 50, 140
    q, k, v = (rnd(s, 1, 2, T, d, dtype=dtype) for s in (8, 9, 10))
    ref, size, reach, _ = oa.window(np64(q), np64(k), np64(v), window, 0, d ** -0.5)
    bound = oa.attention_bound(ref, size, reach, T, d, BITS[dtype], 8 if dtype == BF16 else None)
    k[0, 0, at] = bad
    v[0, 1, at] = bad
    o = lr.lr_fwd_window(q.to(dev), k.to(dev), v.to(dev), window=window)
    torch.cuda.synchronize()
    rows = np.arange(T)
    sees = (rows >= at) & (rows - at < window)
    within(o[:, :, ~torch.from_numpy(sees)], ref[:, :, ~sees], bound[:, :, ~sees])
    got = np64(o)[:, :, sees]
    assert not np.isfinite(got[0, 1]).any()
    if np.isnan(bad):
        assert np.isnan(got[0, 0]).all()


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_window_infinities_and_nan_of_the_values(dev, dtype):
    """A channel with one seen infinity is that infinity, with both signs or a
    NaN it is NaN, and otherwise it is finite, whatever the masked rows beside
    it hold; values near the type's end average without overflow."""
    T, d, window, inf = 200, 64, 40, float("inf")
    q, k, v = (rnd(s, 1, 1, T, d, dtype=dtype) for s in (80, 81, 82))
    ref, size, reach, _ = oa.window(np64(q), np64(k), np64(v), window, 3, d ** -0.5)
    bound = oa.attention_bound(ref, size, reach, T, d, BITS[dtype], 8 if dtype == BF16 else None)
    marks = [(1, 3, inf), (70, 0, inf), (70, 1, -inf), (75, 0, -inf), (80, 2, float("nan")), (90, 2, inf), (150, 5, -inf)]
    for j, ch, x in marks:
        v[0, 0, j, ch] = x
    o = np64(lr.lr_fwd_window(q.to(dev), k.to(dev), v.to(dev), window=window, sinks=3))[0, 0]
    for p in range(T):
        want = {}
        for j, ch, x in marks:
            if oa.sees(p, j, T, window, 3):
                want.setdefault(ch, []).append(x)
        for ch in range(d):
            got = o[p, ch]
            if ch not in want:
                assert abs(got - ref[0, 0, p, ch]) <= bound[0, 0, p, ch], (p, ch, got)
            elif any(np.isnan(x) for x in want[ch]) or len(set(want[ch])) > 1:
                assert np.isnan(got), (p, ch, got)
            else:
                assert got == want[ch][0], (p, ch, got)
    big = torch.finfo(dtype).max / 2
    o = lr.lr_fwd_window(torch.zeros(1, 1, T, d, dtype=dtype, device=dev), k.to(dev),
                         torch.full((1, 1, T, d), big, dtype=dtype, device=dev))
    assert ((o.double() / big - 1).abs() <= 2.0 ** -7).all()


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("which", ["q", "k", "v"])
def test_window_batch_full_of_nan_stays_quick(dev, dtype, which):
    """Everything NaN in one input: every row is NaN, and the call does not
    fall back to a row at a time for each (that took seconds at this size)."""
    import time
    T = 4096
    x = {n: rnd(s, 1, 8, T, 128, dtype=dtype).to(dev) for s, n in ((83, "q"), (84, "k"), (85, "v"))}
    x[which].fill_(float("nan"))
    torch.cuda.synchronize()
    start = time.perf_counter()
    o = lr.lr_fwd_window(x["q"], x["k"], x["v"])
    torch.cuda.synchronize()
    assert time.perf_counter() - start < 1.0
    assert o.isnan().all()


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_window_overlapping_inputs(dev, dtype):
    """Rows that overlap in memory (a sliding view) and one row for all heads."""
    T, d = 140, 64
    line = rnd(86, T * 16 + d, dtype=dtype)
    v = torch.as_strided(line, (1, 2, T, d), (16, 16, 16, 1))
    q, k = (rnd(s, 1, 2, T, d, dtype=dtype) for s in (87, 88))
    dl = line.to(dev)
    o = lr.lr_fwd_window(q.to(dev), k.to(dev), torch.as_strided(dl, (1, 2, T, d), (16, 16, 16, 1)), window=33)
    ref, size, reach, _ = oa.window(np64(q), np64(k), np64(v), 33, 0, d ** -0.5)
    within(o, ref, oa.attention_bound(ref, size, reach, T, d, BITS[dtype], 8 if dtype == BF16 else None))


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_window_extreme_scores(dev, dtype):
    """Scores far beyond exp's range either way, the type's lowest value, and
    -inf: one key decides; equal extremes average; all -inf gives zeros."""
    T, d = 70, 32
    q = torch.zeros(1, 1, T, d, dtype=dtype)
    q[..., 0] = 1
    k = torch.zeros(1, 1, T, d, dtype=dtype)
    v = rnd(11, 1, 1, T, d, dtype=dtype)
    lowest = torch.finfo(dtype).min
    k[0, 0, :, 0] = lowest                      # rows 0..19: all keys alike, at the lowest value
    k[0, 0, 20, 0] = -30000.0                   # from 20 on this one decides
    k[0, 0, 40, 0] = 30000.0                    # from 40 on this one
    ref, size, reach, _ = oa.window(np64(q), np64(k), np64(v), NW, 0, 1.0)
    # products with 0 and 1 are exact here, so the scores are: reach 0
    bound = oa.attention_bound(ref, size, np.zeros_like(reach), T, d, BITS[dtype], 8 if dtype == BF16 else None)
    o = lr.lr_fwd_window(q.to(dev), k.to(dev), v.to(dev), scale=1.0)
    within(o, ref, bound)
    k[0, 0, :, 0] = -float("inf")
    q[...] = 0
    q[..., 0] = 1
    k[..., 1:] = 0
    o = lr.lr_fwd_window(q.to(dev), k.to(dev), v.to(dev), scale=1.0)
    assert (o == 0).all()


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("scale", [0.0, -0.3, 2.5])
def test_window_scales(dev, dtype, scale):
    q, k, v = (rnd(s, 1, 2, 140, 64, dtype=dtype) for s in (12, 13, 14))
    check_window(dev, q, k, v, 77, 2, scale, dtype=dtype)


def _tokens_first(t):
    return t.transpose(1, 2).contiguous().transpose(1, 2)


def _padded(t):
    """Rows with 16 more channels between them, heads and batch swapped in memory."""
    B, H, T, d = t.shape
    big = torch.full((H, B, T, d + 16), float("nan"), dtype=t.dtype, device=t.device)
    view = big.transpose(0, 1)[..., 8 if t.dtype == BF16 else 4:][..., :d]
    view.copy_(t)
    return view


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("views", [_tokens_first, _padded], ids=["tokens-first", "padded"])
@pytest.mark.parametrize("d", [32, 128])
def test_window_strided_tensors(dev, dtype, views, d):
    q, k, v = (rnd(s, 2, h, 150, d, dtype=dtype) for s, h in ((15, 4), (16, 2), (17, 2)))
    check_window(dev, q, k, v, 60, 3, d ** -0.5, dtype=dtype, views=views)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_window_offsets_past_32_bits(dev, dtype):
    """Batches more than 2^31 elements apart in memory."""
    T, d, far = 130, 64, (1 << 31) + 64 * 7
    big = torch.empty(far + 2 * T * d, dtype=dtype, device=dev)
    parts = [rnd(s, 2, 2, T, d, dtype=dtype) for s in (18, 19, 20)]
    def place(t):
        w = torch.as_strided(big, (2, 2, T, d), (far, T * d, d, 1))
        w.copy_(t)
        return w
    q, k, v = parts
    ref, size, reach, _ = oa.window(np64(q), np64(k), np64(v), 50, 2, d ** -0.5)
    bound = oa.attention_bound(ref, size, reach, T, d, BITS[dtype], 8 if dtype == BF16 else None)
    for which in range(3):
        args = [t.to(dev) for t in parts]
        args[which] = place(args[which])
        within(lr.lr_fwd_window(*args, window=50, sinks=2), ref, bound, f"input {which}")
    args = [t.to(dev) for t in parts]
    within(lr.lr_fwd_window(*args, window=50, sinks=2, o=place(torch.zeros_like(args[0]))), ref, bound, "output")


def test_window_lengths_out_of_range_are_reported(dev):
    q, k, v = (rnd(s, 2, 1, 20, 32).to(dev) for s in (21, 22, 23))
    full = lr.lr_fwd_window(q, k, v)
    assert lr.device_status() == LR_OK
    got = lr.lr_fwd_window(q, k, v, k_len=torch.tensor([20, 21], dtype=torch.int32, device=dev))
    assert lr.device_status() == LR_ERR_INDEX and lr.device_status() == LR_OK
    assert torch.equal(got, full)
    o = torch.full_like(q, 7.0)
    lr.lr_fwd_window(q, k, v, q_len=torch.tensor([-3, 400], dtype=torch.int32, device=dev), o=o)
    assert lr.device_status() == LR_ERR_INDEX
    assert (o[0] == 7).all() and torch.equal(o[1], full[1])


def test_window_empty_calls(dev):
    q, k = rnd(24, 2, 2, 0, 64).to(dev), rnd(25, 2, 1, 9, 64).to(dev)
    assert lr.lr_fwd_window(q, k, k).shape == (2, 2, 0, 64)
    q, k = rnd(24, 2, 2, 9, 64, dtype=BF16).to(dev), rnd(25, 2, 1, 0, 64, dtype=BF16).to(dev)
    assert (lr.lr_fwd_window(q, k, k) == 0).all()


# ------------------------------------------------------------------------ step

def paged(seed, lens, Hk, page, d, dtype, dev, garbage=True, extra=2):
    """Pools with the sequences' pages in no order and NaN everywhere else."""
    r = np.random.RandomState(seed)
    need = [max(0, -(-max(L, 0) // page)) for L in lens]
    total, most = sum(need) + extra, max(1, max(need)) + 1
    order = r.permutation(total)
    table = r.randint(0, total, (len(lens), most)).astype(np.int32)
    fill = float("nan") if garbage else 0.0
    kc = torch.full((total, Hk, page, d), fill, dtype=dtype)
    vc = torch.full((total, Hk, page, d), fill, dtype=dtype)
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


def check_step(dev, q, kc, vc, table, lens, window, sinks, scale=None, max_len=None, **kw):
    dtype, d = q.dtype, q.shape[-1]
    scale = d ** -0.5 if scale is None else scale
    o = torch.full(q.shape, 7.0, dtype=dtype, device=dev)
    ld = torch.tensor(lens, dtype=torch.int32, device=dev)
    out = lr.lr_step_paged(q.to(dev), kc, vc, table, ld, max_len=max_len, window=window, sinks=sinks, scale=scale,
                           o=o, **kw)
    torch.cuda.synchronize()
    assert out is o
    ref, size, reach, written = oa.step(np64(q), np64(kc), np64(vc), table.cpu().numpy(), lens, window, sinks, scale)
    bound = oa.attention_bound(ref, size, reach, max(max(lens), 1), d, BITS[dtype], 8 if dtype == BF16 else None)
    w = np.broadcast_to(written[:, None, None], ref.shape)
    within(out, np.where(w, ref, 7.0), np.where(w, bound, 0.0))
    return out


LENS = [1, 0, 15, 16, 17, -1, 127, 128, 129, 300, 601]


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("max_len,window,sinks", [(64, NW, 0), (65, NW, 0), (700, NW, 0), (4096, NW, 0), (4097, NW, 0),
                                                  (20000, 300, 0), (20000, 300, 7), (20000, 4000, 64)])
def test_step_cut_by_the_bound_on_the_length(dev, dtype, max_len, window, sinks):
    """The same short and long sequences under bounds that give one chunk, a
    cluster's few, and many joined by a kernel."""
    lens = [x for x in (1, 0, 64, -1, 63, 700, 4096, 7000) if x <= max_len]
    kc, vc, table = paged(21, lens, 2, 64, 64, dtype, dev)
    wide = torch.zeros(len(lens), -(-max_len // 64), dtype=torch.int32, device=dev)
    most = min(wide.shape[1], table.shape[1])
    wide[:, :most] = table[:, :most]
    check_step(dev, rnd(37, len(lens), 6, 64, dtype=dtype), kc, vc, wide, lens, window, sinks, max_len=max_len)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("d,Hq,Hk", [(32, 8, 8), (128, 8, 2), (64, 17, 1)])
@pytest.mark.parametrize("N", [6, 7, 8, 9, 13, 19, 26, 38])
def test_step_cluster_sizes(dev, dtype, d, Hq, Hk, N):
    """Numbers of sequences that are given to clusters of every size."""
    lens = [(1500 - 41 * i) % 1501 for i in range(N)]
    kc, vc, table = paged(N, lens, Hk, 64, d, dtype, dev)
    check_step(dev, rnd(52, N, Hq, d, dtype=dtype), kc, vc, table, lens, NW, 0)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("Hq,Hk", [(1, 1), (4, 2), (3, 1), (8, 1), (5, 1), (17, 1), (6, 6)])
@pytest.mark.parametrize("page,window,sinks", [(16, NW, 0), (64, 40, 5), (128, 130, 20)])
def test_step_parity(dev, dtype, d, Hq, Hk, page, window, sinks):
    """Lengths of zero, one, page and chunk edges; unused slots; NaN in every
    row of the pools that no sequence holds."""
    kc, vc, table = paged(d + Hq, LENS, Hk, page, d, dtype, dev)
    check_step(dev, rnd(30, len(LENS), Hq, d, dtype=dtype), kc, vc, table, LENS, window, sinks)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (7, 0), (16, 3), (33, 50), (250, 17), (NW, 4)])
@pytest.mark.parametrize("page", [16, 32, 256])
def test_step_sees_each_key_once(dev, dtype, window, sinks, page):
    """Zero keys, values that mark the key (see the window's test)."""
    d, lens = 128, [290, 31, 257]
    kc, vc, table = paged(3, lens, 1, page, d, dtype, dev)
    for n, L in enumerate(lens):
        for j in range(L):
            pg = int(table[n, j // page])
            kc[pg, 0, j % page] = 0
            vc[pg, 0, j % page] = 0
            vc[pg, 0, j % page, j % d] = 1
    check_step(dev, rnd(31, 3, 2, d, dtype=dtype), kc, vc, table, lens, window, sinks, 1.0)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_step_long_cache_is_split_and_joined(dev, dtype):
    """Few sequences, many chunks; the same bits from every call, whatever the
    workspace held, and the bound on the length only changes the cut."""
    lens, d = [5000, 3], 64
    kc, vc, table = paged(5, lens, 1, 64, d, dtype, dev)
    q = rnd(32, 2, 4, d, dtype=dtype)
    a = check_step(dev, q, kc, vc, table, lens, NW, 0, max_len=5000)
    need = lr.step_paged_workspace_size(2, 4, 1, d, 5000, dtype)
    assert need > 0
    ws = torch.full((need,), 255, dtype=torch.uint8, device=dev)
    assert torch.equal(a, check_step(dev, q, kc, vc, table, lens, NW, 0, max_len=5000, workspace=ws))
    assert torch.equal(a, check_step(dev, q, kc, vc, table, lens, NW, 0, max_len=5000, workspace=ws))
    check_step(dev, q, kc, vc, table, lens, NW, 0)
    check_step(dev, q, kc, vc, table, lens, 900, 130)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_step_masked_keys_may_hold_anything(dev, dtype):
    """Keys between the sinks and the window are NaN and infinite."""
    lens, d, page = [400, 131], 128, 32
    kc, vc, table = paged(6, lens, 2, page, d, dtype, dev)
    clean_k, clean_v = kc.clone(), vc.clone()
    for n, L in enumerate(lens):
        for j in range(5, L - 100):
            kc[int(table[n, j // page]), :, j % page] = float("nan") if j % 2 else float("inf")
            vc[int(table[n, j // page]), :, j % page] = float("inf") if j % 3 else float("nan")
    q = rnd(33, 2, 8, d, dtype=dtype)
    a = check_step(dev, q, kc, vc, table, lens, 100, 5)
    b = check_step(dev, q, clean_k, clean_v, table, lens, 100, 5)
    assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_step_non_finite_and_extreme_seen_keys(dev, dtype):
    """A seen NaN makes its heads NaN; -inf scores weigh nothing; only -inf
    scores give zeros; the lowest value everywhere averages."""
    d, lens = 64, [50, 50, 50, 50]
    kc, vc, table = paged(7, lens, 1, 16, d, dtype, dev)
    q = torch.zeros(4, 2, d, dtype=dtype)
    q[..., 0] = 1
    def rows(n):
        return [(int(table[n, j // 16]), j % 16) for j in range(50)]
    for n in range(4):
        for pg, r in rows(n):
            kc[pg, 0, r] = 0
    kc[rows(0)[20][0], 0, rows(0)[20][1], 0] = float("nan")
    for pg, r in rows(1)[1:]:
        kc[pg, 0, r, 0] = -float("inf")
    for pg, r in rows(2):
        kc[pg, 0, r, 0] = -float("inf")
    for pg, r in rows(3):
        kc[pg, 0, r, 0] = torch.finfo(dtype).min
    o = lr.lr_step_paged(q.to(dev), kc, vc, table, torch.tensor(lens, dtype=torch.int32, device=dev), scale=1.0)
    assert o[0].isnan().all() and (o[2] == 0).all()
    first = vc[rows(1)[0][0], 0, rows(1)[0][1]]
    assert torch.equal(o[1, 0], first) and torch.equal(o[1, 1], first)
    mean = np.mean([np64(vc[pg, 0, r]) for pg, r in rows(3)], 0)
    size = np.mean([np.abs(np64(vc[pg, 0, r])) for pg, r in rows(3)], 0)
    bound = oa.attention_bound(mean, size, np.zeros(()), 50, d, BITS[dtype], 8 if dtype == BF16 else None)
    within(o[3, 0], mean, bound)


def test_step_bad_pages_and_lengths_are_reported(dev):
    """A page outside the pool is left out; a length beyond the bound leaves
    its row as it was; both are reported once."""
    lens, d, page = [40, 40, 40], 64, 16
    for dtype in (F32, BF16):
        kc, vc, table = paged(8, lens, 1, page, d, dtype, dev)
        q = rnd(34, 3, 2, d, dtype=dtype).to(dev)
        ld = torch.tensor(lens, dtype=torch.int32, device=dev)
        good = lr.lr_step_paged(q, kc, vc, table, ld)
        assert lr.device_status() == LR_OK
        for bad in (-1, kc.shape[0], 2 ** 31 - 1, -2 ** 31):
            broken = table.clone()
            broken[1, 2] = bad
            o = lr.lr_step_paged(q, kc, vc, broken, ld)
            assert lr.device_status() == LR_ERR_INDEX and lr.device_status() == LR_OK
            assert torch.equal(o[0], good[0]) and torch.equal(o[2], good[2])
            short = torch.tensor([40, 32, 40], dtype=torch.int32, device=dev)
            want, size, reach, _ = oa.step(np64(q), np64(kc), np64(vc), table.cpu().numpy(), [40, 32, 40], NW, 0, d ** -0.5)
            assert lr.lr_step_paged(q, kc, vc, table, short).isfinite().all()
            within(o[1], want[1], oa.attention_bound(want, size, reach, 40, d, BITS[dtype], 8)[1])
        o = torch.full_like(q, 7.0)
        lr.lr_step_paged(q, kc, vc, table, torch.tensor([40, 41, 2 ** 31 - 1], dtype=torch.int32, device=dev),
                         max_len=40, o=o)
        assert lr.device_status() == LR_ERR_INDEX
        assert torch.equal(o[0], good[0]) and (o[1:] == 7).all()
        # the same where chunks are joined by a cluster, and by a second kernel
        for bound_on_len in (300, 20000):
            wide = torch.zeros(3, bound_on_len // page + 1, dtype=torch.int32, device=dev)
            wide[:, :3] = table[:, :3]
            o = torch.full_like(q, 7.0)
            lr.lr_step_paged(q, kc, vc, wide, torch.tensor([40, bound_on_len + 1, -5], dtype=torch.int32, device=dev),
                             max_len=bound_on_len, o=o)
            assert lr.device_status() == LR_ERR_INDEX
            assert torch.equal(o[0], good[0]) and (o[1:] == 7).all()
            wide[0, 1] = -1
            broken = table.clone()
            broken[0, 1] = -1
            a = lr.lr_step_paged(q, kc, vc, wide, ld, max_len=bound_on_len)
            b = lr.lr_step_paged(q, kc, vc, broken, ld)
            assert lr.device_status() == LR_ERR_INDEX
            assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_step_offsets_past_32_bits(dev, dtype):
    """The last pages of a pool of more than 2^31 elements."""
    Hk, page, d = 2, 256, 128
    total = (1 << 31) // (Hk * page * d) + 3
    lens = [520]
    kc, vc, table = paged(9, lens, Hk, page, d, dtype, dev)
    big = [torch.empty(total, Hk, page, d, dtype=dtype, device=dev) for _ in range(2)]
    moved = table.clone()
    for j in range(3):
        moved[0, j] = total - 1 - j
        big[0][total - 1 - j], big[1][total - 1 - j] = kc[int(table[0, j])], vc[int(table[0, j])]
    q = rnd(35, 1, 4, d, dtype=dtype).to(dev)
    ld = torch.tensor(lens, dtype=torch.int32, device=dev)
    assert torch.equal(lr.lr_step_paged(q, *big, moved, ld), lr.lr_step_paged(q, kc, vc, table, ld))


def test_step_sequences_share_pages(dev):
    """Two sequences with the same first pages, and one page used twice by one sequence."""
    d, page = 64, 16
    kc, vc, table = paged(10, [64, 64], 1, page, d, BF16, dev)
    table[1, :2] = table[0, :2]
    table[1, 3] = table[1, 2]
    check_step(dev, rnd(36, 2, 3, d, dtype=BF16), kc, vc, table, [64, 64], NW, 0)


# ------------------------------------------------------------- norm, rotation

def rope_bound(y, size, d, dtype):
    """The norm: a sum of d squares, (d + 3) 2^-24 of it, half of that after
    the root, and four more roundings; cosine and sine: 2^-25 of a half turn
    and two steps, below 2^-21; then the result's rounding."""
    return ((d / 2 + 8) * 2.0 ** -24 + 2.0 ** -21) * size + 2.0 ** -BITS[dtype] * np.abs(y) + 1e-37


ROPE = [  # B, T, Hq, Hk, d, rot, interleaved, norm, weights
    (1, 1, 1, 1, 32, 32, False, True, True), (2, 5, 4, 2, 64, 64, False, True, True),
    (1, 33, 3, 1, 128, 128, False, True, True), (2, 17, 6, 2, 128, 128, True, True, False),
    (1, 40, 2, 2, 64, 32, False, True, True), (1, 40, 2, 2, 64, 16, True, False, False),
    (3, 7, 5, 5, 128, 48, False, False, False), (1, 9, 8, 1, 128, 96, False, True, True),
    (1, 129, 4, 4, 32, 16, False, True, False), (2, 3, 9, 3, 64, 0, False, True, True),
    (1, 6, 2, 1, 32, 0, False, False, False), (64, 1, 8, 2, 128, 128, False, True, True),
    (1, 700, 16, 4, 128, 128, False, True, True),
]


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("case", ROPE, ids=lambda c: "-".join(str(int(x)) for x in c))
@pytest.mark.parametrize("append", [False, True], ids=["plain", "append"])
def test_norm_rope_parity(dev, case, dtype, append):
    """Views of one projection as inputs; positions from 0 to an int's end and
    padding; outputs and, with a cache, exactly the rows of the positions."""
    B, T, Hq, Hk, d, rot, inter, norm, weights = case
    x = rnd(40, B, T, Hq + 2 * Hk, d, dtype=dtype)
    q, k, v = (x[:, :, a:b].transpose(1, 2) for a, b in ((0, Hq), (Hq, Hq + Hk), (Hq + Hk, Hq + 2 * Hk)))
    xd = x.to(dev)
    qd, kd, vd = (xd[:, :, a:b].transpose(1, 2) for a, b in ((0, Hq), (Hq, Hq + Hk), (Hq + Hk, Hq + 2 * Hk)))
    r = np.random.RandomState(T)
    page = 16
    if append:  # distinct positions over a few pages
        span = 4 * page * (1 + T // (3 * page))
        pos = np.stack([r.permutation(span)[:T] for _ in range(B)]).astype(np.int32)
    else:
        pos = r.choice([0, 1, 7, 4095, 131071, 1000003, 2 ** 31 - 1], (B, T)).astype(np.int32)
    if T > 1:
        pos[r.rand(B, T) < 0.2] = -1
    pd = torch.from_numpy(pos).to(dev)
    qw, kw = (rnd(s, d) for s in (41, 42)) if weights else (None, None)
    f = None
    if rot:
        f = torch.from_numpy(10000.0 ** (-np.arange(rot // 2) / (rot // 2)))
    kwargs = {}
    if append:
        most = -(-span // page)
        total = B * most + 1
        table = torch.from_numpy(r.permutation(total)[:B * most].reshape(B, most).astype(np.int32)).to(dev)
        kc, vc = (torch.full((total, Hk, page, d), 7.0, dtype=dtype, device=dev) for _ in range(2))
        kwargs = dict(v=vd, k_cache=kc, v_cache=vc, table=table)
    qo = torch.full((B, Hq, T, d), 7.0, dtype=dtype, device=dev)
    ko = torch.full((B, Hk, T, d), 7.0, dtype=dtype, device=dev)
    dw = [None if w is None else w.to(dev) for w in (qw, kw)]
    got = lr.lr_qk_norm_rope(qd, kd, pd, norm=norm, q_weight=dw[0], k_weight=dw[1], eps=1e-5,
                             inv_freq=None if f is None else f.to(dev), interleaved=inter, q_out=qo, k_out=ko, **kwargs)
    torch.cuda.synchronize()
    assert got[0] is qo and got[1] is ko
    keep = np.broadcast_to((pos >= 0)[:, None, :, None], qo.shape)
    for t, out, w in ((q, qo, qw), (k, ko, kw)):
        y, size = oa.qk_norm_rope(np64(t), pos, None if w is None else np64(w), 1e-5 if norm else None,
                                  None if f is None else f.numpy(), inter)
        kp = keep[:, :1]
        within(out, np.where(kp, y, 7.0), np.where(kp, rope_bound(y, size, d, dtype), 0.0))
    if append:
        wk, wv = (torch.full((total, Hk, page, d), 7.0, dtype=dtype) for _ in range(2))
        tb, kh = table.cpu(), ko.cpu()
        for b in range(B):
            for t in range(T):
                p = int(pos[b, t])
                if p >= 0:
                    wk[tb[b, p // page], :, p % page] = kh[b, :, t]
                    wv[tb[b, p // page], :, p % page] = v[b, :, t]
        assert torch.equal(kc.cpu(), wk) and torch.equal(vc.cpu(), wv)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("d,B,T", [(128, 3, 1), (64, 2, 90), (32, 4, 3000)])
def test_norm_rope_long_padding(dev, dtype, d, B, T):
    """Whole stretches of padding: what is computed behind and before them is
    as it is without them, and the padded rows stay as they were."""
    q, k = (rnd(s, B, h, T, d, dtype=dtype).to(dev) for s, h in ((46, 5), (47, 2)))
    f = torch.tensor(10000.0 ** (-np.arange(d // 2) / (d // 2)), device=dev)
    pos = torch.arange(T, dtype=torch.int32, device=dev).expand(B, T).contiguous()
    want = lr.lr_qk_norm_rope(q, k, pos, inv_freq=f)
    pos[0] = -1
    pos[1, T // 3:T // 3 * 2 + 1] = -1
    got = (torch.full_like(want[0], 7.0), torch.full_like(want[1], 7.0))
    lr.lr_qk_norm_rope(q, k, pos, inv_freq=f, q_out=got[0], k_out=got[1])
    for g, w in zip(got, want):
        on = (pos >= 0)[:, None, :, None]
        assert torch.equal(g, torch.where(on, w, torch.full_like(w, 7.0)))


def test_norm_rope_default_positions_and_cache_only_keys(dev):
    B, T, d, page = 2, 37, 64, 16
    q, k, v = (rnd(s, B, h, T, d, dtype=BF16).to(dev) for s, h in ((43, 4), (44, 2), (45, 2)))
    f = torch.tensor(10000.0 ** (-np.arange(32) / 32), device=dev)
    pos = torch.arange(T, dtype=torch.int32, device=dev).expand(B, T).contiguous()
    want = lr.lr_qk_norm_rope(q, k, pos, inv_freq=f)
    got = lr.lr_qk_norm_rope(q, k, inv_freq=f)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    table = torch.arange(6, dtype=torch.int32, device=dev).view(2, 3)
    kc, vc = (torch.zeros(6, 2, page, d, dtype=BF16, device=dev) for _ in range(2))
    qo, none = lr.lr_qk_norm_rope(q, k, inv_freq=f, v=v, k_cache=kc, v_cache=vc, table=table, write_k=False)
    assert none is None and torch.equal(qo, want[0])
    flat = lambda c: c.view(2, 3, 2, page, d).transpose(1, 2).reshape(2, 2, 48, d)[:, :, :T]
    assert torch.equal(flat(kc), want[1]) and torch.equal(flat(vc), v)


def test_norm_rope_bad_pages_are_reported(dev):
    """A page outside the pool or a position behind the table writes nothing
    to the cache, is reported, and leaves the contiguous outputs as they are."""
    d, page = 64, 16
    q, k, v = (rnd(s, 1, 1, 3, d).to(dev) for s in (46, 47, 48))
    want = lr.lr_qk_norm_rope(q, k)[1]
    for pos, entry in (((0, 16, 5), -1), ((0, 17, 5), 4), ((0, 32, 5), 1), ((0, 2 ** 31 - 1, 5), 1)):
        table = torch.tensor([[2, entry]], dtype=torch.int32, device=dev)
        kc, vc = (torch.full((4, 1, page, d), 7.0, device=dev) for _ in range(2))
        pd = torch.tensor([pos], dtype=torch.int32, device=dev)
        ko = lr.lr_qk_norm_rope(q, k, pd, v=v, k_cache=kc, v_cache=vc, table=table)[1]
        assert lr.device_status() == LR_ERR_INDEX and lr.device_status() == LR_OK
        assert torch.equal(ko, want)
        left = torch.full_like(kc, 7.0)
        left[2, 0, 0], left[2, 0, 5] = want[0, 0, 0], want[0, 0, 2]
        assert torch.equal(kc, left)


# ----------------------------------------------------- together, streams, graphs

@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("window,sinks", [(24, 3), (None, 0)])
def test_prompt_then_steps_together(dev, dtype, window, sinks):
    """A layer's life: the prompts of a padded batch through norm, rotation,
    append and window attention, then tokens one by one through append and the
    paged step; every output row against the definition over the whole
    sequence, with the keys as the first operator stored them."""
    B, Hq, Hk, d, page, steps = 3, 4, 2, 64, 16, 5
    T, lens = 50, [50, 17, 1]
    w = NW if window is None else window
    x = rnd(50, B, T + steps, Hq + 2 * Hk, d, dtype=dtype).to(dev)
    split = lambda y: [y[:, :, a:b].transpose(1, 2) for a, b in ((0, Hq), (Hq, Hq + Hk), (Hq + Hk, Hq + 2 * Hk))]
    f = torch.tensor(10000.0 ** (-np.arange(d // 2) / (d // 2)), device=dev)
    most = -(-(T + steps) // page)
    table = torch.randperm(B * most, generator=torch.Generator().manual_seed(1)).int().view(B, most).to(dev)
    kc, vc = (torch.full((B * most, Hk, page, d), float("nan"), dtype=dtype, device=dev) for _ in range(2))
    cache = dict(k_cache=kc, v_cache=vc, table=table)
    pos = torch.arange(T).repeat(B, 1)
    pos[pos >= torch.tensor(lens)[:, None]] = -1
    q, k, v = split(x[:, :T])
    ld = torch.tensor(lens, dtype=torch.int32, device=dev)
    qo, ko = lr.lr_qk_norm_rope(q, k, pos.int().to(dev), inv_freq=f, v=v, **cache)
    o = lr.lr_fwd_window(qo, ko, v, window=window, sinks=sinks, q_len=ld, k_len=ld)
    outs, qs = [o], [qo]
    for s in range(steps):
        qn, kn, vn = split(x[:, T + s:T + s + 1])
        p = (ld + s).view(B, 1)
        qo, _ = lr.lr_qk_norm_rope(qn, kn, p, inv_freq=f, v=vn, write_k=False, **cache)
        outs.append(lr.lr_step_paged(qo.view(B, Hq, d), kc, vc, table, ld + s + 1, window=window, sinks=sinks,
                                     max_len=T + steps))
        qs.append(qo)
    torch.cuda.synchronize()
    kn, vn, tn = np64(kc), np64(vc), table.cpu().numpy()
    wb = 8 if dtype == BF16 else None
    for b in range(B):
        L = lens[b] + steps
        rows = (tn[b, np.arange(L) // page], slice(None), np.arange(L) % page)
        keys, vals = kn[rows].transpose(1, 0, 2)[None], vn[rows].transpose(1, 0, 2)[None]
        query = np.concatenate([np64(qs[0])[b, :, :lens[b]]] + [np64(y)[b] for y in qs[1:]], 1)[None]
        got = torch.cat([outs[0][b, :, :lens[b]]] + [y[b].unsqueeze(1) for y in outs[1:]], 1)[None]
        ref, size, reach, _ = oa.window(query, keys, vals, w, sinks, d ** -0.5)
        within(got, ref, oa.attention_bound(ref, size, reach, L, d, BITS[dtype], wb), f"sequence {b}")


def test_operators_capture_into_graphs_and_follow_their_inputs(dev):
    """One graph of append + step replayed as its lengths, positions and
    inputs change; a second graph shares the workspace on the same stream."""
    B, Hq, Hk, d, page, most = 2, 4, 1, 128, 16, 400
    f = torch.tensor(10000.0 ** (-np.arange(64) / 64), device=dev)
    table = torch.arange(B * most, dtype=torch.int32, device=dev).view(B, most)
    kc, vc = (rnd(s, B * most, Hk, page, d, dtype=BF16).to(dev) for s in (60, 61))
    x = rnd(62, B, 1, Hq + 2 * Hk, d, dtype=BF16).to(dev)
    pos = torch.tensor([[5900], [4]], dtype=torch.int32, device=dev)
    lens = torch.tensor([5901, 5], dtype=torch.int32, device=dev)
    ws = torch.empty(lr.step_paged_workspace_size(B, Hq, Hk, d, most * page, BF16), dtype=torch.uint8, device=dev)
    assert ws.numel() > 0

    def once(window):
        q, k, v = (x[:, :, a:b].transpose(1, 2) for a, b in ((0, Hq), (Hq, Hq + Hk), (Hq + Hk, Hq + 2 * Hk)))
        qo, _ = lr.lr_qk_norm_rope(q, k, pos, inv_freq=f, v=v, k_cache=kc, v_cache=vc, table=table, write_k=False)
        return lr.lr_step_paged(qo.view(B, Hq, d), kc, vc, table, lens, window=window, workspace=ws)

    ws2 = lr.step_paged_workspace_size(B, Hq, Hk, d, most * page, BF16, window=700)
    assert ws2 <= ws.numel()
    once(None), once(700)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for window in (None, 700):   # chunks joined by a kernel, and by a cluster
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(once(window))
        graphs.append(g)
    for s in range(3):
        x.copy_(rnd(63 + s, *x.shape, dtype=BF16))
        for i, window in ((0, None), (1, 700), (0, None)):
            outs[i].fill_(7.0)
            graphs[i].replay()
            assert torch.equal(outs[i], once(window))
        pos += 1
        lens += 1


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_window_captures_into_a_graph(dev, dtype):
    """Replays follow inputs and lengths; more pieces of work than SMs."""
    B, T = 3, 700
    q, k, v = (rnd(s, B, h, T, 64, dtype=dtype).to(dev) for s, h in ((90, 16), (91, 8), (92, 8)))
    ql = torch.tensor([700, 300, 5], dtype=torch.int32, device=dev)
    kl = ql.clone()
    call = lambda: lr.lr_fwd_window(q, k, v, window=130, sinks=4, q_len=ql, k_len=kl)
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o = call()
    for s in range(3):
        q.copy_(rnd(93 + s, *q.shape, dtype=dtype))
        g.replay()
        assert torch.equal(o, call())
        ql -= 2
        kl -= 1


def test_two_calls_at_once(dev):
    """Two streams run the three operators at the same time: the same bits as alone."""
    q, k, v = (rnd(s, 2, h, 3000, 128, dtype=BF16).to(dev) for s, h in ((96, 8), (97, 8), (98, 8)))
    f = torch.tensor(10000.0 ** (-np.arange(64) / 64), device=dev)
    kc, vc, table = paged(12, [4000] * 3, 2, 64, 128, BF16, dev)
    lens = torch.tensor([4000] * 3, dtype=torch.int32, device=dev)
    x = rnd(99, 3, 8, 128, dtype=BF16).to(dev)

    def three(window):
        a, b = lr.lr_qk_norm_rope(q, k, inv_freq=f)
        return a, b, lr.lr_fwd_window(a, b, v, window=window), lr.lr_step_paged(x, kc, vc, table, lens, window=window)

    want = [three(None), three(500)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(dev) for _ in range(2)]
    for _ in range(3):
        got = []
        for s, w in zip(streams, (None, 500)):
            with torch.cuda.stream(s):
                got.append(three(w))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_operators_on_another_stream_and_repeated(dev):
    """Calls given a stream run there (their outputs too), and repeated calls
    give the same bits."""
    q, k, v = (rnd(s, 2, h, 600, 128, dtype=BF16).to(dev) for s, h in ((70, 4), (71, 2), (72, 2)))
    kc, vc, table = paged(11, [3000, 40], 2, 64, 128, BF16, dev)
    lens = torch.tensor([3000, 40], dtype=torch.int32, device=dev)
    qs = q[:, :, 0].contiguous()
    def all_three(stream=None):
        a, b = lr.lr_qk_norm_rope(q, k, stream=stream)
        return (a, b, lr.lr_fwd_window(a, b, v, window=200, sinks=4, stream=stream),
                lr.lr_step_paged(qs, kc, vc, table, lens, stream=stream))
    want = all_three()
    torch.cuda.synchronize()
    side = torch.cuda.Stream(dev)
    for _ in range(3):
        got = all_three(side)
        side.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))
    with torch.cuda.stream(side):
        got = all_three()
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))


def _scores_of_one_channel(scores, heads, rows, d, dtype, dev):
    """q, k [1,heads,..,d] whose products are exactly `scores` (two bf16 parts
    a key) for every row."""
    q = torch.zeros(1, heads, rows, d, dtype=dtype)
    q[..., :2] = 1
    k = torch.zeros(1, heads, len(scores[0]), d, dtype=dtype)
    k[..., 0], k[..., 1] = (torch.tensor(s, dtype=torch.float64).to(dtype) for s in scores)
    return q.to(dev), k.to(dev)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("H", [1, 160], ids=["cluster", "alone"])
@pytest.mark.parametrize("scale", [1.0, 2.5, -1.0])
@pytest.mark.parametrize("top", [2.0 ** 33, 2.0 ** 40, 2.0 ** 66, 2.0 ** 126, None], ids=lambda t: f"{t or 'max'}")
def test_window_large_finite_scores(dev, top, scale, H, dtype):
    """Scores from 1e10 to the type's largest: those alike share the weight,
    and one that is a 64th part above them takes all of it."""
    d, Tq, Tk, at = 32, 30, 700, 685
    top = torch.finfo(dtype).max if top is None else top
    key = np.full(Tk, top * (1 - 2.0 ** -6))
    key[at] = top
    q, k = _scores_of_one_channel((key * np.sign(scale), np.zeros(Tk)), H, Tq, d, dtype, dev)
    v = rnd(120, 1, 1, Tk, d, dtype=dtype)
    o = lr.lr_fwd_window(q, k, v.expand(1, H, Tk, d).contiguous().to(dev), scale=scale)
    ref, size, reach, _ = oa.window(np64(q[:, :1]), np64(k[:, :1]), np64(v), NW, 0, scale)
    # products with 0 and 1 are exact, so the scores are: reach 0
    bound = oa.attention_bound(ref, size, np.zeros_like(reach), Tk, d, BITS[dtype], 8 if dtype == BF16 else None)
    within(o, np.broadcast_to(ref, o.shape), np.broadcast_to(bound, o.shape))


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("H", [1, 160], ids=["cluster", "alone"])
@pytest.mark.parametrize("base", [1.8125, 1.46875, -1.8125])
def test_window_weights_of_tiles_agree_at_large_scores(dev, base, H, dtype):
    """512 keys and, in a later tile, one that is 7 above them: the weights of
    both tiles refer to the same maximum, however large the scores are.  These
    are exact in fp32 (2^21 and small integers), and what the exponential takes
    is below 32, so its roundings are those of scores of that size."""
    d, Tq, Tk, at = 32, 30, 700, 660
    big, small = np.full(Tk, base * 2.0 ** 21), np.zeros(Tk)
    small[512:] = -100.0
    small[at] = 7.0
    q, k = _scores_of_one_channel((big, small), H, Tq, d, dtype, dev)
    v = torch.ones(1, H, Tk, d, dtype=dtype)
    v[:, :, at] = -1
    o = lr.lr_fwd_window(q, k, v.to(dev), scale=1.0)
    ref, size, reach, _ = oa.window(np64(q[:, :1]), np64(k[:, :1]), np64(v[:, :1]), NW, 0, 1.0)
    bound = oa.attention_bound(ref, size, np.full_like(reach, 32.0), Tk, d, BITS[dtype], 8 if dtype == BF16 else None)
    within(o, np.broadcast_to(ref, o.shape), np.broadcast_to(bound, o.shape))


STEP_CUTS = [64, 700, 40000]   # bounds on the length: one chunk, a cluster's few, many joined by a kernel


def _wide(table, max_len, page, dev):
    """The table with room for max_len tokens (page 0 where the sequences end)."""
    wide = torch.zeros(table.shape[0], -(-max_len // page), dtype=torch.int32, device=dev)
    most = min(wide.shape[1], table.shape[1])
    wide[:, :most] = table[:, :most]
    return wide


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("d,Hq,Hk", [(32, 2, 1), (64, 17, 1), (128, 6, 2)])
@pytest.mark.parametrize("max_len", STEP_CUTS)
def test_step_values_that_are_not_finite_or_overflow_a_sum(dev, max_len, d, Hq, Hk, dtype):
    """The step's row is the window's: a channel with a seen infinity is that
    infinity (of a key whose weight underflows, too), with both signs or a NaN
    it is NaN, any other is as without them; values near the type's end average
    without overflow; a page outside the pool is left out of all this."""
    page, inf, lens = 16, float("inf"), [50, 61, 64, 33, 40]
    kc, vc, table = paged(130, lens, Hk, page, d, dtype, dev)
    q = rnd(131, len(lens), Hq, d, dtype=dtype)
    place = lambda n, j: (int(table[n, j // page]), slice(None), j % page)
    q[0] = 1
    kc[place(0, 9)] = -1e4                     # score -1e4 sqrt(d): no weight
    for n, j in ((2, j) for j in range(lens[2])):
        vc[place(n, j)] = torch.finfo(dtype).max / 2
    ref, size, reach, _ = oa.step(np64(q), np64(kc), np64(vc), table.cpu().numpy(), lens, NW, 0, d ** -0.5)
    marks = [(0, 9, 3, inf), (0, 9, 5, -inf), (1, 0, 1, inf), (1, 60, 1, -inf), (1, 17, 2, float("nan")),
             (1, 31, 4, -inf), (1, 32, 4, -inf), (4, 3, 0, inf)]
    want, bound = ref.copy(), oa.attention_bound(ref, size, reach, 64, d, BITS[dtype], 8 if dtype == BF16 else None)
    # sequence 4: its second page is outside the pool
    left = [j for j in range(lens[4]) if j // page != 1]
    rows = (table[4].cpu().numpy()[np.array(left) // page], slice(None), np.array(left) % page)
    for h in range(Hq):
        a, s, r = oa.row(np64(q)[4, h], np64(kc)[rows][:, h // (Hq // Hk)], np64(vc)[rows][:, h // (Hq // Hk)], d ** -0.5)
        want[4, h], bound[4, h] = a, oa.attention_bound(a, s, np.array(r), 64, d, BITS[dtype], 8 if dtype == BF16 else None)
    for n, j, ch, x in marks:
        vc[place(n, j)][:, ch] = x
    wide = _wide(table, max_len, page, dev)
    wide[4, 1] = kc.shape[0]
    need = lr.step_paged_workspace_size(len(lens), Hq, Hk, d, max_len, dtype)
    assert (need > 0) == (max_len == STEP_CUTS[2])
    o = lr.lr_step_paged(q.to(dev), kc, vc, wide, torch.tensor(lens, dtype=torch.int32, device=dev), max_len=max_len)
    assert lr.device_status() == LR_ERR_INDEX
    got = np64(o)
    for n, ch, x in ((0, 3, inf), (0, 5, -inf), (1, 1, np.nan), (1, 2, np.nan), (1, 4, -inf), (4, 0, inf)):
        assert np.array_equal(got[n, :, ch], np.full(Hq, x), equal_nan=True), (n, ch, got[n, :, ch])
        got[n, :, ch] = want[n, :, ch] = 0
    within(torch.from_numpy(got), want, bound)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("which", ["k", "v"])
def test_step_batch_full_of_nan_stays_quick(dev, which, dtype):
    """Every row NaN: found from a few keys, not by a row at a time over all."""
    import time
    N, L, page = 64, 4096, 64
    pools = {n: rnd(132, N * L // page, 2, page, 64, dtype=dtype).to(dev) for n in ("k", "v")}
    pools[which].fill_(float("nan"))
    table = torch.arange(N * L // page, dtype=torch.int32, device=dev).view(N, -1)
    q, lens = rnd(133, N, 8, 64, dtype=dtype).to(dev), torch.full((N,), L, dtype=torch.int32, device=dev)
    torch.cuda.synchronize()
    start = time.perf_counter()
    o = lr.lr_step_paged(q, pools["k"], pools["v"], table, lens)
    torch.cuda.synchronize()
    assert time.perf_counter() - start < 1.0
    assert o.isnan().all()


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("scale", [0.0, -0.3, 2.5])
@pytest.mark.parametrize("max_len", STEP_CUTS)
def test_step_scales(dev, max_len, scale, dtype):
    lens = [64, 1, 17, 0, 33]
    kc, vc, table = paged(134, lens, 2, 16, 64, dtype, dev)
    wide = _wide(table, max_len, 16, dev)
    check_step(dev, rnd(135, len(lens), 6, 64, dtype=dtype), kc, vc, wide, lens, NW, 0, scale, max_len=max_len)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("scale", [0.0, -0.3, 2.5])
def test_window_scales_of_few_rows_and_many_keys(dev, scale, dtype):
    q, k, v = (rnd(s, 1, 2, t, 64, dtype=dtype) for s, t in ((136, 17), (137, 1500), (138, 1500)))
    check_window(dev, q, k, v, NW, 0, scale, dtype=dtype)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_scale_of_zero_averages_whatever_the_scores_are(dev, dtype):
    """q . k from the type's lowest to its largest value: times zero all alike."""
    d, T = 64, 60
    q = torch.zeros(1, 2, T, d, dtype=dtype)
    q[..., 0] = 1
    k = rnd(139, 1, 2, T, d, dtype=dtype)
    k[..., 0] = torch.finfo(dtype).max / 4 * k[..., 0].float().clamp(-4, 4).to(dtype)
    k[:, :, 5, 0], k[:, :, 6, 0] = torch.finfo(dtype).min, torch.finfo(dtype).max
    v = rnd(140, 1, 2, T, d, dtype=dtype)
    ref, size, reach, _ = oa.window(np64(q), np64(k), np64(v), NW, 0, 0.0)
    bound = oa.attention_bound(ref, size, np.zeros_like(reach), T, d, BITS[dtype], 8 if dtype == BF16 else None)
    within(lr.lr_fwd_window(q.to(dev), k.to(dev), v.to(dev), scale=0.0), ref, bound, "window")
    for H in (1, 160):   # few rows: a cluster's parts, and alone
        big = [t[:, :1].expand(1, H, T, d).repeat(1, 1, 12, 1).contiguous().to(dev) for t in (k, v)]
        o = lr.lr_fwd_window(q[:, :1, :9].expand(1, H, 9, d).contiguous().to(dev), *big, scale=0.0)
        a, s, _, _ = oa.window(np64(q[:, :1, :9]), *(np64(t[:, :1]) for t in big), NW, 0, 0.0)
        b = oa.attention_bound(a, s, np.zeros(a.shape[:3]), 12 * T, d, BITS[dtype], 8 if dtype == BF16 else None)
        within(o, np.broadcast_to(a, o.shape), np.broadcast_to(b, o.shape), f"window, {H} heads")
    pool = lambda t: torch.cat((t, torch.zeros(1, 2, 4, d, dtype=dtype)), 2).view(2, 4, 16, d).transpose(0, 1).contiguous().to(dev)
    table = torch.arange(4, dtype=torch.int32, device=dev).view(1, 4)
    for max_len in STEP_CUTS:
        o = lr.lr_step_paged(q[:, :, -1].contiguous().to(dev), pool(k), pool(v), _wide(table, max_len, 16, dev),
                             torch.tensor([T], dtype=torch.int32, device=dev), max_len=max_len, scale=0.0)
        within(o, ref[:, :, -1], bound[:, :, -1], f"step, {max_len}")


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_scales_at_the_ends_of_fp32(dev, dtype):
    """The largest scale leaves the largest score alone, the smallest averages."""
    d, T = 32, 50
    q, k, v = (rnd(s, 1, 1, T, d, dtype=dtype) for s in (141, 142, 143))
    for scale in (3.4e38, -3.4e38, 1e-44):
        ref, size, reach, _ = oa.window(np64(q), np64(k), np64(v), NW, 0, scale)
        # the scores of these seeds are far enough apart for fp32 to order them
        bound = oa.attention_bound(ref, size, np.zeros_like(reach), T, d, BITS[dtype], 8 if dtype == BF16 else None)
        within(lr.lr_fwd_window(q.to(dev), k.to(dev), v.to(dev), scale=scale), ref, bound, f"window, {scale}")
        pool = lambda t: torch.cat((t, torch.zeros(1, 1, 14, d, dtype=dtype)), 2).view(4, 1, 16, d).to(dev)
        o = lr.lr_step_paged(q[:, :, -1].contiguous().to(dev), pool(k), pool(v),
                             torch.arange(4, dtype=torch.int32, device=dev).view(1, 4),
                             torch.tensor([T], dtype=torch.int32, device=dev), scale=scale)
        within(o, ref[:, :, -1], bound[:, :, -1], f"step, {scale}")


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("d,B,T,Hq,Hk", [(128, 3, 1, 4, 1), (64, 2, 90, 5, 2), (32, 4, 3000, 3, 1)])
def test_norm_rope_own_outputs_are_zero_in_the_padding(dev, d, B, T, Hq, Hk, dtype):
    """Outputs that the call makes have zeros where nothing is computed,
    whatever their memory held, and the other rows as in given outputs."""
    q, k, v = (rnd(s, B, h, T, d, dtype=dtype).to(dev) for s, h in ((150, Hq), (151, Hk), (152, Hk)))
    f = torch.tensor(10000.0 ** (-np.arange(d // 2) / (d // 2)), device=dev)
    pos = torch.arange(T, dtype=torch.int32, device=dev).expand(B, T).contiguous()
    pos[0] = -1
    pos[1, T // 3:T // 3 * 2 + 1] = -5
    most = -(-T // 16)
    cache = dict(v=v, table=torch.arange(B * most, dtype=torch.int32, device=dev).view(B, most))
    for write_k in (True, False):
        kc, vc = (torch.full((B * most, Hk, 16, d), 7.0, dtype=dtype, device=dev) for _ in range(2))
        want = [torch.full_like(q, 7.0), torch.full_like(k, 7.0)]
        lr.lr_qk_norm_rope(q, k, pos, inv_freq=f, q_out=want[0], k_out=want[1], k_cache=kc, v_cache=vc, **cache)
        pools = [kc.clone(), vc.clone()]
        on = (pos >= 0)[:, None, :, None]
        junk = [torch.full_like(t, float("nan")) for t in (q, k, q, k)]
        del junk   # what the allocator hands out next
        got = lr.lr_qk_norm_rope(q, k, pos, inv_freq=f, write_k=write_k, k_cache=kc, v_cache=vc, **cache)
        assert torch.equal(got[0], torch.where(on, want[0], torch.zeros_like(q)))
        assert got[1] is None if not write_k else torch.equal(got[1], torch.where(on, want[1], torch.zeros_like(k)))
        assert torch.equal(kc, pools[0]) and torch.equal(vc, pools[1])
    junk = [torch.full_like(t, float("nan")) for t in (q, k)]
    given, junk = junk[0], None   # one output given, one made
    got = lr.lr_qk_norm_rope(q, k, pos, inv_freq=f, q_out=given.fill_(7.0))
    assert torch.equal(given, want[0]) and torch.equal(got[1], torch.where(on, want[1], torch.zeros_like(k)))


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("d,Hq,Hk", [(32, 3, 3), (64, 17, 1), (128, 8, 2)])
@pytest.mark.parametrize("max_len", STEP_CUTS)
def test_step_own_output_is_zero_in_unused_slots(dev, max_len, d, Hq, Hk, dtype):
    """The same for unused slots and lengths beyond the bound."""
    lens = [64, -1, 17, max_len + 1, -2 ** 31, 3]
    kc, vc, table = paged(153, [64, 0, 17, 0, 0, 3], Hk, 16, d, dtype, dev)
    wide = _wide(table, max_len, 16, dev)
    q, ld = rnd(154, len(lens), Hq, d, dtype=dtype).to(dev), torch.tensor(lens, dtype=torch.int32, device=dev)
    want = lr.lr_step_paged(q, kc, vc, wide, ld, max_len=max_len, o=torch.zeros_like(q))
    junk = [torch.full_like(q, float("nan")) for _ in range(4)]
    del junk
    got = lr.lr_step_paged(q, kc, vc, wide, ld, max_len=max_len)
    assert lr.device_status() == LR_ERR_INDEX
    assert torch.equal(got, want) and (got[[1, 3, 4]] == 0).all() and (got[[0, 2, 5]] != 0).any()


@pytest.mark.parametrize("Hq,Hk", [(70000, 1), (3, 40000)])
def test_norm_rope_of_many_heads(dev, Hq, Hk):
    q, k = (rnd(s, 1, h, 1, 32, dtype=BF16) for s, h in ((160, Hq), (161, Hk)))
    got = lr.lr_qk_norm_rope(q.to(dev), k.to(dev), eps=1e-5)
    for t, out in ((q, got[0]), (k, got[1])):
        y, size = oa.qk_norm_rope(np64(t), np.zeros((1, 1)), None, 1e-5)
        within(out, y, rope_bound(y, size, 32, BF16))


def _turned(x, p, f):
    """x [d] turned in split halves by p f, the angle reduced in rationals."""
    from fractions import Fraction
    turn = 2 * Fraction(3141592653589793238462643383279502884197169399375105820974944592, 10 ** 63)
    th = np.array([float(p * Fraction(y) % turn) for y in f])
    a, b = x[:len(f)], x[len(f):]
    c, s = np.cos(th), np.sin(th)
    return np.concatenate((a * c - b * s, b * c + a * s)), np.tile(np.abs(a) + np.abs(b), 2)


@pytest.mark.parametrize("interleaved", [False, True])
def test_norm_rope_fast_angles_at_far_positions(dev, interleaved):
    """Radians per position of any size, at positions up to an int's end."""
    f = np.array([6.1, -2.9, 1e3 / 7, -1.0 / 3, 2.0 ** 40 / 3, 1e-30, -1e-30, 0.0, 3.0, 5.5, 1.0, 0.7, 40.0, -77.7, 1e6 / 3, 2.0])
    pos = np.array([1, 2 ** 31 - 1, 2 ** 31 - 2, 1000003, 131071, 0], np.int32)
    x = rnd(162, 1, 1, len(pos), 32)
    x[0, 0] = x[0, 0, 0]
    laid = x[..., torch.arange(32).view(2, 16).T.reshape(-1)] if interleaved else x
    got = lr.lr_qk_norm_rope(laid.to(dev), laid.to(dev), torch.from_numpy(pos)[None].to(dev), norm=False,
                             inv_freq=torch.from_numpy(f).to(dev), interleaved=interleaved)[0].cpu()
    if interleaved:
        got = torch.cat((got[..., 0::2], got[..., 1::2]), -1)
    for i, p in enumerate(pos):
        y, size = _turned(np64(x[0, 0, i]), int(p), f)
        within(got[0, 0, i], y, rope_bound(y, size, 32, F32), f"position {p}")


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("sign", [1, -1])
def test_means_of_values_at_the_end_of_the_type_are_finite(dev, sign, d, dtype):
    """Every value the type's largest: whatever the weights round to, the mean
    is that value, and no rounding of it may leave the type."""
    top = sign * torch.finfo(dtype).max
    for B, Hq, Hk, Tq, Tk in ((1, 160, 160, 40, 300), (1, 2, 1, 40, 700), (1, 3, 1, 9, 200)):
        q, k = (rnd(s, B, h, t, d, dtype=dtype).to(dev) for s, h, t in ((170, Hq, Tq), (171, Hk, Tk)))
        v = torch.full((B, Hk, Tk, d), top, dtype=dtype, device=dev)
        o = lr.lr_fwd_window(q, k, v, window=250, sinks=2)
        assert ((o.double() / top - 1).abs() <= 2.0 ** -7).all()
    lens = [64, 1, 17, 50]
    kc, vc, table = paged(172, lens, 1, 16, d, dtype, dev)
    vc.fill_(top)
    q, ld = rnd(173, len(lens), 8, d, dtype=dtype).to(dev), torch.tensor(lens, dtype=torch.int32, device=dev)
    for max_len in STEP_CUTS:
        o = lr.lr_step_paged(q, kc, vc, _wide(table, max_len, 16, dev), ld, max_len=max_len)
        assert ((o.double() / top - 1).abs() <= 2.0 ** -7).all()
