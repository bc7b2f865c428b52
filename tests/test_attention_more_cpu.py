"""CPU-side checks of the rotation by several axes, of differential attention and
of the step over a shared prefix: refusals before any launch and the binding's
checks."""
import os
import subprocess
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

_START = r"""
import ctypes, sys
sys.path.insert(0, sys.argv[1])
import gated_delta_rule_fwd_gb300 as lr
from gated_delta_rule_fwd_gb300.attention import Strides, Paged, QkMaps, DiffMaps
L = lr.lib()
A = [0x10000000 * (i + 1) for i in range(16)]   # distinct, aligned, never dereferenced
P = lambda a: None if a is None else ctypes.c_void_p(a)
def contig(H, T, d): return (H * T * d, T * d, d)
inf, nan = float('inf'), float('nan')
"""
_END = r"""
bad = [(n, got, want) for n, got, want in cases if got != want]
print("BAD", bad)
sys.exit(1 if bad else 0)
"""

_AXES = r"""
def axes(**kw):
    a = dict(q=A[0], k=A[1], pos=A[2], qo=A[3], ko=A[4], v=A[5], ck=A[6], cv=A[7], tab=A[8], qw=A[9], kw=A[10],
             f=A[11], axis=A[12], places=A[13], axes=3, flags=1, eps=1e-6, rot=32, pages=4, page=16, most=4,
             B=2, T=5, Hq=4, Hk=2, d=64, dt=1, cache=True, maps=True, qs=None, ks=None, vs=None)
    a.update(kw)
    S = lambda s, H: Strides(*(s or contig(H, max(a['T'], 1), a['d'])))
    m = QkMaps(a['flags'], a['qw'], a['kw'], a['eps'], a['rot'], a['f'])
    c = Paged(a['ck'], a['cv'], a['tab'], a['pages'], a['page'], a['most'])
    return L.lr_qk_norm_rope_axes(P(a['q']), S(a['qs'], a['Hq']), P(a['k']), S(a['ks'], a['Hk']), P(a['pos']),
                                  P(a['axis']), a['axes'], P(a['places']), ctypes.byref(m) if a['maps'] else None,
                                  P(a['qo']), P(a['ko']), P(a['v']), S(a['vs'], a['Hk']),
                                  ctypes.byref(c) if a['cache'] else None, a['B'], a['T'], a['Hq'], a['Hk'],
                                  a['d'], a['dt'], None)
cases = [
    ("ok", axes(), 7), ("nocache-ok", axes(cache=False, v=None), 7), ("places-null-ok", axes(places=None), 7),
    ("T0", axes(T=0, q=None), 0), ("axes0", axes(axes=0), 2), ("axes-neg", axes(axes=-3), 2),
    ("axes16-ok", axes(axes=16), 7), ("axes17", axes(axes=17), 2),
    ("null-axis", axes(axis=None), 1), ("null-pos", axes(pos=None), 1), ("no-rotation-ok", axes(axis=None, pos=None, f=None, rot=0), 7),
    ("align-axis", axes(axis=A[12] + 2), 4), ("align-axis-ok", axes(axis=A[12] + 4), 7), ("align-pos", axes(pos=A[2] + 1), 4),
    ("align-places", axes(places=A[13] + 2), 4),
    ("alias-axis", axes(qo=A[12]), 8), ("alias-pos", axes(ko=A[2]), 8),
    # the last axis's positions, 2 x 5 x 4 bytes an axis
    ("alias-pos-last", axes(ko=A[2] + 112), 8), ("alias-pos-behind-ok", axes(ko=A[2] + 128), 7),
    ("alias-places", axes(qo=A[13]), 8), ("alias-unused-axis", axes(qo=A[12], rot=0), 7),
    ("dtype", axes(dt=2), 3), ("d48", axes(d=48), 6), ("flag", axes(flags=4), 12), ("rot-odd", axes(rot=24), 6),
    ("null-maps", axes(maps=False), 1), ("null-freq", axes(f=None), 1), ("null-v", axes(v=None), 1),
    ("page", axes(page=24), 6), ("stride-odd", axes(qs=(1280, 320, 68)), 4), ("alias-qo-q", axes(qo=A[0]), 8),
]
"""


_DIFF = r"""
def diff(**kw):
    a = dict(q=A[0], k=A[1], v=A[2], ql=A[3], kl=A[4], o=A[5], lam=A[6], w=A[7], ws=A[8], wsb=1 << 26, flags=1,
             eps=1e-6, B=2, H=4, Hk=2, Tq=5, Tk=9, d=64, win=4, s=1, scale=0.5, dt=1, qs=None, ks=None, vs=None,
             os=None, maps=True)
    a.update(kw)
    S = lambda s, H, T: Strides(*(s or contig(2 * H, max(T, 1), a['d'])))
    m = DiffMaps(a['flags'], a['lam'], a['w'], a['eps'])
    return L.lr_fwd_diff(P(a['q']), S(a['qs'], a['H'], a['Tq']), P(a['k']), S(a['ks'], a['Hk'], a['Tk']),
                         P(a['v']), S(a['vs'], a['Hk'], a['Tk']), P(a['ql']), P(a['kl']),
                         ctypes.byref(m) if a['maps'] else None, P(a['o']), S(a['os'], a['H'], a['Tq']),
                         a['B'], a['H'], a['Hk'], a['Tq'], a['Tk'], a['d'], a['win'], a['s'], a['scale'], a['dt'],
                         P(a['ws']), a['wsb'], None)
wsz = lambda *a: L.lr_fwd_diff_workspace_size(*a)
need = wsz(2, 4, 2, 5, 9, 64, 0)
cases = [
    ("ok", diff(), 7), ("f32-ok", diff(dt=0), 7), ("Tq0", diff(Tq=0, q=None), 0), ("Tk0-ok", diff(Tk=0, k=None, v=None), 7),
    ("dtype", diff(dt=-1), 3), ("d256", diff(d=256), 6), ("d16", diff(d=16), 6), ("heads", diff(H=5), 2), ("Hk0", diff(Hk=0), 2),
    ("window0", diff(win=0), 2), ("sinks", diff(s=-1), 2), ("scale", diff(scale=inf), 2), ("B0", diff(B=0), 2),
    ("Tneg", diff(Tk=-1), 2), ("huge", diff(Tq=1 << 30, B=1 << 10), 2), ("many", diff(H=1 << 30, Hk=1 << 30), 2),
    ("null-maps", diff(maps=False), 1), ("null-lam", diff(lam=None), 1), ("null-w-ok", diff(w=None), 7),
    ("flag", diff(flags=2), 12), ("eps", diff(eps=-1.0), 12), ("eps-nan", diff(eps=nan), 12), ("eps-unused", diff(flags=0, eps=nan), 7),
    ("null-q", diff(q=None), 1), ("null-k", diff(k=None), 1), ("null-o", diff(o=None), 1), ("null-len-ok", diff(ql=None, kl=None), 7),
    ("align-v", diff(v=A[2] + 4), 4), ("align-len", diff(kl=A[4] + 1), 4), ("align-lam", diff(lam=A[6] + 2), 4),
    ("align-lam-ok", diff(lam=A[6] + 4), 7), ("align-w", diff(w=A[7] + 1), 4),
    ("stride-k0", diff(ks=(2304, 0, 64)), 2), ("stride-odd", diff(vs=(2304, 576, 60)), 4),
    ("o-rows-overlap", diff(os=(2560, 320, 32)), 8), ("o-tokens-first-ok", diff(os=(2560, 64, 512)), 7),
    ("alias-q", diff(o=A[0] + 1024), 8), ("alias-len", diff(o=A[3] - 1024), 8), ("alias-lam", diff(o=A[6]), 8),
    ("alias-w", diff(o=A[7]), 8), ("alias-w-unused", diff(o=A[7], flags=0), 7),
    ("ws-null", diff(dt=0, ws=None), 10), ("ws-short", diff(dt=0, wsb=need - 1), 10), ("ws-align", diff(dt=0, ws=A[8] + 8), 4),
    ("ws-alias-o", diff(dt=0, ws=A[5]), 8), ("ws-alias-q", diff(dt=0, ws=A[0]), 8), ("ws-unused-ok", diff(ws=None, wsb=0), 7),
    ("ws-need", int(need > 0), 1), ("ws-bf16", wsz(2, 4, 2, 5, 9, 64, 1), 0), ("ws-bad", wsz(2, 4, 3, 5, 9, 64, 0), 0),
]
"""


_DIFF_STEP = r"""
def step(**kw):
    a = dict(q=A[0], ck=A[1], cv=A[2], tab=A[3], lens=A[4], o=A[5], lam=A[6], w=A[7], ws=A[8], wsb=1 << 27, flags=1,
             eps=1e-6, N=3, H=4, Hk=2, d=64, most_len=9000, win=1 << 30, s=0, scale=0.5, dt=1, pages=9, page=16,
             most=600, cache=True, maps=True)
    a.update(kw)
    c = Paged(a['ck'], a['cv'], a['tab'], a['pages'], a['page'], a['most'])
    m = DiffMaps(a['flags'], a['lam'], a['w'], a['eps'])
    return L.lr_step_paged_diff(P(a['q']), ctypes.byref(c) if a['cache'] else None, P(a['lens']),
                                ctypes.byref(m) if a['maps'] else None, P(a['o']), a['N'], a['H'], a['Hk'], a['d'],
                                a['most_len'], a['win'], a['s'], a['scale'], a['dt'], P(a['ws']), a['wsb'], None)
wsz = lambda *a: L.lr_step_paged_diff_workspace_size(*a)
need = wsz(3, 4, 2, 64, 9000, 1 << 30, 0, 1)
cases = [
    ("ok", step(), 7), ("f32-ok", step(dt=0), 7), ("fill-ok", step(flags=3), 7), ("flag", step(flags=4), 12),
    ("dtype", step(dt=9), 3), ("d16", step(d=16), 6), ("N0", step(N=0), 2), ("heads", step(H=3), 2),
    ("window", step(win=0), 2), ("sinks", step(s=-2), 2), ("scale", step(scale=nan), 2), ("maxlen0", step(most_len=0), 2),
    ("maxlen-table", step(most_len=16 * 600 + 1), 2), ("null-lens", step(lens=None), 1), ("null-cache", step(cache=False), 1),
    ("null-pool", step(cv=None), 1), ("null-maps", step(maps=False), 1), ("null-lam", step(lam=None), 1),
    ("null-w-ok", step(w=None), 7), ("page", step(page=512), 6), ("eps", step(eps=inf), 12),
    ("align-o", step(o=A[5] + 8), 4), ("align-lam", step(lam=A[6] + 2), 4), ("alias-q", step(o=A[0]), 8),
    ("alias-pool", step(o=A[2] + 64), 8), ("alias-lam", step(o=A[6]), 8), ("alias-w", step(o=A[7]), 8),
    # the pools hold 2 Hk heads: 9 x 4 x 16 x 64 x 2 bytes
    ("alias-pool-end", step(o=A[2] + 9 * 4 * 16 * 64 * 2 - 16), 8), ("alias-pool-behind-ok", step(o=A[2] + 9 * 4 * 16 * 64 * 2), 7),
    ("ws-null", step(ws=None), 10), ("ws-short", step(wsb=need - 1), 10), ("ws-align", step(ws=A[8] + 8), 4),
    ("ws-alias", step(ws=A[5]), 8), ("many", step(N=1 << 30, H=4, Hk=4), 2),
    ("ws-split", int(need > 0), 1), ("ws-one-chunk", wsz(3, 4, 2, 64, 64, 1 << 30, 0, 1), 0),
    ("ws-cluster", wsz(3, 4, 2, 64, 300, 1 << 30, 0, 1), 0), ("ws-bad", wsz(3, 4, 3, 64, 300, 1, 0, 1), 0),
]
"""


_PREFIX = r"""
def step(**kw):
    a = dict(q=A[0], ck=A[1], cv=A[2], tab=A[3], lens=A[4], o=A[5], pre=A[6], P=1000, ws=A[8], wsb=1 << 27, flags=0,
             N=3, Hq=4, Hk=2, d=64, most_len=9000, win=1 << 30, s=0, scale=0.5, dt=1, pages=9, page=16, most=600,
             cache=True)
    a.update(kw)
    c = Paged(a['ck'], a['cv'], a['tab'], a['pages'], a['page'], a['most'])
    return L.lr_step_paged_prefix(P(a['q']), ctypes.byref(c) if a['cache'] else None, P(a['pre']), a['P'], P(a['lens']),
                                  P(a['o']), a['N'], a['Hq'], a['Hk'], a['d'], a['most_len'], a['win'], a['s'],
                                  a['scale'], a['flags'], a['dt'], P(a['ws']), a['wsb'], None)
wsz = lambda *a: L.lr_step_paged_prefix_workspace_size(*a)
need = wsz(3, 4, 2, 64, 1000, 9000, 1 << 30, 0, 1)
cases = [
    ("ok", step(), 7), ("f32-ok", step(dt=0), 7), ("fill-ok", step(flags=1), 7), ("flag", step(flags=2), 12),
    ("P0-ok", step(P=0, pre=None), 7), ("P-neg", step(P=-1), 2), ("P-long", step(P=1 << 30), 2),
    ("P-longest-ok", step(P=(1 << 30) - 9000, win=5, wsb=1 << 40), 7),
    ("null-prefix", step(pre=None), 1), ("align-prefix", step(pre=A[6] + 2), 4), ("align-prefix-ok", step(pre=A[6] + 4), 7),
    ("alias-prefix", step(o=A[6]), 8), ("alias-prefix-end", step(o=A[6] + 240), 8), ("alias-prefix-behind-ok", step(o=A[6] + 256), 7),
    ("ws-alias-prefix", step(ws=A[6]), 8), ("ws-alias-o", step(ws=A[5]), 8),
    ("dtype", step(dt=9), 3), ("d16", step(d=16), 6), ("N0", step(N=0), 2), ("heads", step(Hq=3), 2), ("window", step(win=0), 2),
    ("sinks", step(s=-2), 2), ("scale", step(scale=nan), 2), ("maxlen0", step(most_len=0), 2),
    ("maxlen-table", step(most_len=16 * 600 + 1), 2), ("null-lens", step(lens=None), 1), ("null-cache", step(cache=False), 1),
    ("null-pool", step(cv=None), 1), ("page", step(page=512), 6), ("align-o", step(o=A[5] + 8), 4),
    ("alias-q", step(o=A[0]), 8), ("alias-pool", step(o=A[2] + 64), 8), ("many", step(N=1 << 30, Hq=4, Hk=4), 2),
    ("ws-null", step(ws=None), 10), ("ws-short", step(wsb=need - 1), 10), ("ws-align", step(ws=A[8] + 8), 4),
    ("ws-need", int(need > 0), 1), ("ws-none", wsz(3, 4, 2, 64, 0, 64, 1 << 30, 0, 1), 0),
    ("ws-left-behind", wsz(3, 4, 2, 64, 100000, 64, 1 << 30, 0, 1) > wsz(3, 4, 2, 64, 100000, 64, 50, 0, 1) > 0, True),
    ("ws-bad", wsz(3, 4, 3, 64, 100, 300, 1, 0, 1), 0),
]
"""


def _child(body):
    from gated_delta_rule_fwd_gb300.build import build
    build()
    env = dict(os.environ, CUDA_VISIBLE_DEVICES="")
    r = subprocess.run([sys.executable, "-c", _START + body + _END, ROOT], env=env, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr


def test_axes_arguments_rejected_before_launch():
    """In a child without a GPU: a call that passes validation then fails at
    its launch (LR_ERR_CUDA, 7)."""
    _child(_AXES)


def test_diff_arguments_rejected_before_launch():
    _child(_DIFF)


def test_diff_step_arguments_rejected_before_launch():
    _child(_DIFF_STEP)


def test_prefix_arguments_rejected_before_launch():
    _child(_PREFIX)


def test_struct_sizes_match_the_header():
    import ctypes
    from gated_delta_rule_fwd_gb300 import attention as at
    src = ('#include "lr_attn.h"\n'
           f"_Static_assert(sizeof(lr_diff_maps) == {ctypes.sizeof(at.DiffMaps)}, \"maps\");\n"
           f"_Static_assert(LR_MAX_AXES == {at.MAX_AXES} && LR_DIFF_NORM == {at.DIFF_NORM}, \"values\");\n"
           f"_Static_assert(LR_DIFF_FILL == {at.DIFF_FILL} && LR_STEP_FILL == {at.STEP_FILL}, \"values\");\n"
           "int main(void) { return 0; }\n")
    inc = [a for d in ("/usr/local/cuda/include",) if os.path.isdir(d) for a in ("-I", d)]
    r = subprocess.run(["gcc", "-std=c11", "-fsyntax-only", "-x", "c", "-I", os.path.join(ROOT, "include"),
                        *inc, "-"], input=src, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


class _NoLaunch:
    def __getattr__(self, name):
        raise AssertionError(f"the binding reached the library ({name}) with invalid arguments")


@pytest.fixture
def lr(monkeypatch):
    import gated_delta_rule_fwd_gb300 as lr
    monkeypatch.setattr(lr, "_require_cuda", lambda dev: None)   # CPU tensors stand in
    monkeypatch.setattr(torch.cuda, "current_device", lambda: None)
    monkeypatch.setattr(lr, "lib", lambda: _NoLaunch())
    return lr


def _t(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype)


def _i(*shape, dtype=torch.int32):
    return torch.zeros(*shape, dtype=dtype)


def _axes_args(**change):
    a = dict(q=_t(2, 4, 9, 64), k=_t(2, 2, 9, 64), positions=_i(3, 2, 9), axis=_i(32), places=_i(2, 9),
             inv_freq=torch.zeros(32, dtype=torch.float64))
    a.update(change)
    return a


def test_axes_binding_accepts_what_it_should(lr):
    for change in (dict(), dict(places=None), dict(positions=_i(1, 2, 9)), dict(inv_freq=None, axis=_i(0))):
        with pytest.raises(AssertionError, match="lr_qk_norm_rope_axes"):
            lr.lr_qk_norm_rope_axes(**_axes_args(**change))


@pytest.mark.parametrize("change", [
    dict(positions=None), dict(axis=None), dict(positions=_i(2, 9)), dict(positions=_i(3, 2, 8)),
    dict(positions=_i(17, 2, 9)), dict(positions=_i(0, 2, 9)), dict(positions=_i(3, 2, 9, dtype=torch.int64)),
    dict(positions=_i(2, 9, 3).permute(2, 0, 1)), dict(axis=_i(31)), dict(axis=_i(32, dtype=torch.int64)),
    dict(axis=_i(64)[::2]), dict(places=_i(9)), dict(places=_i(2, 9, dtype=torch.int64)), dict(inv_freq=None),
    dict(v=_t(2, 2, 9, 64)), dict(write_k=False), dict(k=_t(2, 2, 8, 64))], ids=lambda c: "-".join(c))
def test_axes_binding_refuses(lr, change):
    with pytest.raises((ValueError, TypeError)):
        lr.lr_qk_norm_rope_axes(**_axes_args(**change))


def _diff_args(**change):
    a = dict(q=_t(1, 4, 9, 64), k=_t(1, 2, 9, 64), v=_t(1, 2, 9, 64), lam=torch.zeros(2))
    a.update(change)
    return a


def test_diff_binding_accepts_what_it_should(lr):
    for change in (dict(), dict(norm=False), dict(norm_weight=torch.zeros(128)), dict(q_len=_i(1), k_len=_i(1))):
        with pytest.raises(AssertionError, match="lr_fwd_diff"):
            lr.lr_fwd_diff(**_diff_args(**change))


@pytest.mark.parametrize("change", [
    dict(q=_t(1, 3, 9, 64)), dict(k=_t(1, 3, 9, 64)), dict(k=_t(1, 2, 9, 32)), dict(v=_t(1, 2, 8, 64)), dict(v=_t(1, 1, 9, 128)),
    dict(q=_t(4, 9, 64)), dict(q=_t(1, 4, 64, 9).transpose(2, 3)), dict(lam=torch.zeros(4)), dict(lam=_t(2)),
    dict(lam=torch.zeros(4)[::2]), dict(norm_weight=torch.zeros(64)), dict(norm=False, norm_weight=torch.zeros(128)),
    dict(q_len=_i(1, dtype=torch.int64)), dict(k_len=_i(2)), dict(o=_t(1, 4, 9, 32)), dict(window=1 << 40),
    dict(q=_t(1, 4, 9, 64, dtype=torch.float16))], ids=lambda c: "-".join(c))
def test_diff_binding_refuses(lr, change):
    with pytest.raises((ValueError, TypeError)):
        lr.lr_fwd_diff(**_diff_args(**change))


def _diff_step_args(**change):
    a = dict(q=_t(3, 4, 64), k_cache=_t(5, 2, 16, 64), v_cache=_t(5, 2, 16, 64), table=_i(3, 4), lens=_i(3),
             lam=torch.zeros(2))
    a.update(change)
    return a


def test_diff_step_binding_accepts_what_it_should(lr):
    for change in (dict(max_len=60), dict(norm=False), dict(norm_weight=torch.zeros(128))):
        with pytest.raises(AssertionError, match="lr_step_paged_diff"):
            lr.lr_step_paged_diff(**_diff_step_args(**change))


@pytest.mark.parametrize("change", [
    dict(q=_t(3, 3, 64)), dict(k_cache=_t(5, 3, 16, 64), v_cache=_t(5, 3, 16, 64)), dict(q=_t(1, 3, 4, 64)),
    dict(v_cache=_t(5, 1, 16, 128)), dict(table=_i(2, 4)), dict(lens=_i(4)), dict(lens=None), dict(lam=torch.zeros(3)),
    dict(lam=None), dict(norm=False, norm_weight=torch.zeros(128)), dict(o=_t(3, 4, 32)), dict(max_len=1 << 33)],
    ids=lambda c: "-".join(c))
def test_diff_step_binding_refuses(lr, change):
    with pytest.raises((ValueError, TypeError, AttributeError)):
        lr.lr_step_paged_diff(**_diff_step_args(**change))


def _prefix_args(**change):
    a = dict(q=_t(3, 4, 64), k_cache=_t(5, 2, 16, 64), v_cache=_t(5, 2, 16, 64), prefix=_i(4), prefix_len=50,
             table=_i(3, 4), lens=_i(3))
    a.update(change)
    return a


def test_prefix_binding_accepts_what_it_should(lr):
    for change in (dict(max_len=60), dict(prefix_len=64), dict(prefix=_i(0), prefix_len=0)):
        with pytest.raises(AssertionError, match="lr_step_paged_prefix"):
            lr.lr_step_paged_prefix(**_prefix_args(**change))


@pytest.mark.parametrize("change", [
    dict(prefix=None), dict(prefix=_i(3)), dict(prefix=_i(1, 4)), dict(prefix=_i(4, dtype=torch.int64)), dict(prefix=_i(8)[::2]),
    dict(prefix_len=65), dict(prefix_len=1 << 40), dict(q=_t(1, 3, 4, 64)), dict(v_cache=_t(5, 1, 16, 128)), dict(table=_i(2, 4)),
    dict(lens=_i(4)), dict(lens=None), dict(o=_t(3, 4, 32)), dict(max_len=1 << 33)], ids=lambda c: "-".join(c))
def test_prefix_binding_refuses(lr, change):
    with pytest.raises((ValueError, TypeError)):
        lr.lr_step_paged_prefix(**_prefix_args(**change))
