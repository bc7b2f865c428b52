"""lr_qk_norm_rope_axes against its fp64 definition (oracle/attention.py),
element by element within a derived bound, and against lr_qk_norm_rope where
the two agree by definition.
"""
import numpy as np
import pytest
import torch

import gated_delta_rule_fwd_gb300 as lr
from oracle import attention as oa

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
BITS = {F32: 24, BF16: 8}          # half a step of the type, 2^-bits relative
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


def freqs(half, dev, base=10000.0):
    return torch.tensor(base ** (-np.arange(half) / half), dtype=torch.float64, device=dev)


def ints(x, dev):
    return torch.from_numpy(np.ascontiguousarray(x).astype(np.int32)).to(dev)


def bound_of(y, size, d, dtype):
    """The norm: a sum of d squares, (d + 3) 2^-24 of it, half of that after
    the root, and four more roundings; cosine and sine: 2^-25 of a half turn
    and two steps, below 2^-21; the definition's own angles: fp64 products of up
    to 2^31 radians, 2^-22; then the result's rounding."""
    return ((d / 2 + 8) * 2.0 ** -24 + 2.0 ** -21 + 2.0 ** -22) * size + 2.0 ** -BITS[dtype] * np.abs(y) + 1e-37


def within(got, want, bound):
    got = np64(got)
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), (f"{bad.sum()} of {bad.size} outside, first at {np.argwhere(bad)[0]}: "
                           f"{got[bad][0]} for {want[bad][0]} +- {bound[bad][0]}")


CASES = [  # B, T, Hq, Hk, d, rot, interleaved, norm, weights, axes, axis of the pairs: runs or in turn
    (1, 1, 1, 1, 32, 32, False, True, True, 3, "runs"), (2, 5, 4, 2, 64, 64, False, True, True, 2, "turn"),
    (1, 33, 3, 1, 128, 128, True, True, True, 3, "turn"), (2, 17, 6, 2, 128, 128, False, True, False, 4, "runs"),
    (1, 40, 2, 2, 64, 32, False, True, True, 3, "runs"), (1, 40, 2, 2, 64, 16, True, False, False, 16, "turn"),
    (3, 7, 5, 5, 128, 48, False, False, False, 1, "runs"), (1, 129, 4, 4, 32, 16, False, True, False, 2, "turn"),
    (2, 3, 9, 3, 64, 0, False, True, True, 2, "runs"), (64, 1, 8, 2, 128, 128, False, True, True, 3, "runs"),
    (1, 700, 16, 4, 128, 128, False, True, True, 3, "turn"),
]


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(x if isinstance(x, str) else int(x)) for x in c))
@pytest.mark.parametrize("append", [False, True], ids=["plain", "append"])
def test_axes_parity(dev, case, dtype, append):
    """Views of one projection as inputs; positions over the whole range of an
    int; places of their own and padding; with a cache, exactly the rows of the
    places."""
    B, T, Hq, Hk, d, rot, inter, norm, weights, axes, how = case
    x = rnd(40, B, T, Hq + 2 * Hk, d, dtype=dtype)
    cut = ((0, Hq), (Hq, Hq + Hk), (Hq + Hk, Hq + 2 * Hk))
    q, k, v = (x[:, :, a:b].transpose(1, 2) for a, b in cut)
    xd = x.to(dev)
    qd, kd, vd = (xd[:, :, a:b].transpose(1, 2) for a, b in cut)
    r = np.random.RandomState(T)
    page, half = 16, rot // 2
    pos = r.choice([0, 1, 7, 4095, 131071, 1000003, 2 ** 31 - 1, -1, -1000, -2 ** 31], (axes, B, T))
    axis = np.arange(half) * axes // max(half, 1) if how == "runs" else np.arange(half) % axes
    span = 4 * page * (1 + T // (3 * page))
    place = np.stack([r.permutation(span)[:T] for _ in range(B)])
    if T > 1:
        place[r.rand(B, T) < 0.2] = -1
    qw, kw = (rnd(s, d) for s in (41, 42)) if weights else (None, None)
    f = freqs(half, dev) if half else None
    kwargs = {}
    if append:
        most = -(-span // page)
        total = B * most + 1
        table = ints(r.permutation(total)[:B * most].reshape(B, most), dev)
        kc, vc = (torch.full((total, Hk, page, d), 7.0, dtype=dtype, device=dev) for _ in range(2))
        kwargs = dict(v=vd, k_cache=kc, v_cache=vc, table=table)
    qo = torch.full((B, Hq, T, d), 7.0, dtype=dtype, device=dev)
    ko = torch.full((B, Hk, T, d), 7.0, dtype=dtype, device=dev)
    dw = [None if w is None else w.to(dev) for w in (qw, kw)]
    got = lr.lr_qk_norm_rope_axes(qd, kd, ints(pos, dev), ints(axis, dev), ints(place, dev), norm=norm,
                                  q_weight=dw[0], k_weight=dw[1], eps=1e-5, inv_freq=f, interleaved=inter,
                                  q_out=qo, k_out=ko, **kwargs)
    torch.cuda.synchronize()
    assert got[0] is qo and got[1] is ko
    keep = (place >= 0)[:, None, :, None]
    for t, out, w in ((q, qo, qw), (k, ko, kw)):
        y, size = oa.qk_norm_rope_axes(np64(t), pos, axis, None if w is None else np64(w), 1e-5 if norm else None,
                                       None if f is None else np64(f), inter)
        on = np.broadcast_to(keep, y.shape)
        within(out, np.where(on, y, 7.0), np.where(on, bound_of(y, size, d, dtype), 0.0))
    if append:
        wk, wv = (torch.full((total, Hk, page, d), 7.0, dtype=dtype) for _ in range(2))
        tb, kh = table.cpu(), ko.cpu()
        for b in range(B):
            for t in range(T):
                p = int(place[b, t])
                if p >= 0:
                    wk[tb[b, p // page], :, p % page] = kh[b, :, t]
                    wv[tb[b, p // page], :, p % page] = v[b, :, t]
        assert torch.equal(kc.cpu(), wk) and torch.equal(vc.cpu(), wv)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("d,B,T", [(128, 3, 1), (64, 2, 90), (32, 4, 3000)])
def test_axes_that_agree_are_one_axis(dev, dtype, d, B, T):
    """The same positions on every axis: the bits of lr_qk_norm_rope; outputs
    that the call makes are zeros in the padding."""
    q, k = (rnd(s, B, h, T, d, dtype=dtype).to(dev) for s, h in ((46, 5), (47, 2)))
    f = freqs(d // 2, dev)
    pos = torch.arange(T, dtype=torch.int32, device=dev).expand(B, T).contiguous()
    want = lr.lr_qk_norm_rope(q, k, pos, inv_freq=f)
    three = pos.expand(3, B, T).contiguous()
    axis = (torch.arange(d // 2, device=dev) % 3).int()
    got = lr.lr_qk_norm_rope_axes(q, k, three, axis, inv_freq=f)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    places = pos.clone()
    places[0, T // 2:] = -1
    got = lr.lr_qk_norm_rope_axes(q, k, three, axis, places, inv_freq=f)
    on = (places >= 0)[:, None, :, None]
    assert all(torch.equal(a, torch.where(on, b, torch.zeros_like(b))) for a, b in zip(got, want))


def test_axes_default_places_and_keys_in_the_cache_only(dev):
    B, T, d, page = 2, 37, 64, 16
    q, k, v = (rnd(s, B, h, T, d, dtype=BF16).to(dev) for s, h in ((43, 4), (44, 2), (45, 2)))
    f, axis = freqs(32, dev), (torch.arange(32, device=dev) % 2).int()
    pos = torch.randint(0, 99, (2, B, T), device=dev).int()
    want = lr.lr_qk_norm_rope_axes(q, k, pos, axis, inv_freq=f)
    table = torch.arange(6, dtype=torch.int32, device=dev).view(2, 3)
    kc, vc = (torch.zeros(6, 2, page, d, dtype=BF16, device=dev) for _ in range(2))
    qo, none = lr.lr_qk_norm_rope_axes(q, k, pos, axis, inv_freq=f, v=v, k_cache=kc, v_cache=vc, table=table,
                                       write_k=False)
    assert none is None and torch.equal(qo, want[0])
    flat = lambda c: c.view(2, 3, 2, page, d).transpose(1, 2).reshape(2, 2, 48, d)[:, :, :T]
    assert torch.equal(flat(kc), want[1]) and torch.equal(flat(vc), v)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_axes_bad_axis_and_bad_pages_are_reported(dev, dtype):
    """A pair whose axis is out of range is turned by axis 0; a place without a
    page is written nowhere; both are reported."""
    d, page = 64, 16
    q, k, v = (rnd(s, 1, 1, 3, d, dtype=dtype).to(dev) for s in (46, 47, 48))
    f, axis = freqs(32, dev), torch.zeros(32, dtype=torch.int32, device=dev)
    axis[5:9] = 1
    pos = torch.tensor([[[3, 5, 9]], [[1, 0, 4]]], dtype=torch.int32, device=dev)
    want = lr.lr_qk_norm_rope_axes(q, k, pos, axis, inv_freq=f)
    assert lr.device_status() == LR_OK
    for bad in (-1, 2, 2 ** 31 - 1, -2 ** 31):
        broken = axis.clone()
        broken[20] = bad
        got = lr.lr_qk_norm_rope_axes(q, k, pos, broken, inv_freq=f)
        assert lr.device_status() == LR_ERR_INDEX and lr.device_status() == LR_OK
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    # without a rotation neither is read
    lr.lr_qk_norm_rope_axes(q, k, pos, axis[:0])
    assert lr.device_status() == LR_OK
    for places, entry in (((0, 16, 5), -1), ((0, 17, 5), 4), ((0, 32, 5), 1), ((0, 2 ** 31 - 1, 5), 1)):
        table = torch.tensor([[2, entry]], dtype=torch.int32, device=dev)
        kc, vc = (torch.full((4, 1, page, d), 7.0, dtype=dtype, device=dev) for _ in range(2))
        ko = lr.lr_qk_norm_rope_axes(q, k, pos, axis, torch.tensor([places], dtype=torch.int32, device=dev), inv_freq=f,
                                     v=v, k_cache=kc, v_cache=vc, table=table)[1]
        assert lr.device_status() == LR_ERR_INDEX and lr.device_status() == LR_OK
        assert torch.equal(ko, want[1])
        left = torch.full_like(kc, 7.0)
        left[2, 0, 0], left[2, 0, 5] = want[1][0, 0, 0], want[1][0, 0, 2]
        assert torch.equal(kc, left)


def test_axes_capture_and_another_stream(dev):
    """A captured call follows its inputs; a call on a stream of its own gives the same bits."""
    B, T, d = 3, 50, 128
    q, k = (rnd(s, B, h, T, d, dtype=BF16).to(dev) for s, h in ((51, 4), (52, 2)))
    f, axis = freqs(64, dev), (torch.arange(64, device=dev) // 22).int()
    pos = torch.randint(0, 500, (3, B, T), device=dev).int()
    call = lambda **kw: lr.lr_qk_norm_rope_axes(q, k, pos, axis, inv_freq=f, **kw)
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = call()
    for s in range(3):
        q.copy_(rnd(53 + s, *q.shape, dtype=BF16))
        pos += 1
        g.replay()
        want = call()
        assert all(torch.equal(a, b) for a, b in zip(out, want))
    side = torch.cuda.Stream(dev)
    torch.cuda.synchronize()
    got = call(stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
