"""CPU-side checks of the attention entry points (include/lr_attn.h): symbols,
refusals before any launch, the binding's checks."""
import os
import re
import subprocess
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "lr_attn.h")


@pytest.fixture(scope="module")
def lib():
    from gated_delta_rule_fwd_gb300.build import build
    build()
    import gated_delta_rule_fwd_gb300 as lr
    return lr.lib()


def _declared():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    return sorted(set(re.findall(r"\b(lr_[a-z_]+)\s*\(", text)))


def test_entry_points_declared_exported_and_bound(lib):
    import gated_delta_rule_fwd_gb300 as lr
    assert tuple(_declared()) == tuple(sorted(lr.ATTN_SYMBOLS))
    out = subprocess.run(["nm", "-D", "--defined-only", lib._name], capture_output=True, text=True,
                         check=True).stdout
    exported = set(re.findall(r"\sT\s+(\w+)", out))
    for name in _declared():
        assert name in exported
    assert callable(lr.lr_qk_norm_rope) and callable(lr.lr_fwd_window) and callable(lr.lr_step_paged)
    assert lr.status_string(13) == "a page or a length on the device is out of range"


def test_headers_compile_as_c_and_struct_sizes_match():
    import ctypes
    from gated_delta_rule_fwd_gb300 import attention as at
    src = ('#include "lr_attn.h"\n'
           f"_Static_assert(sizeof(lr_strides) == {ctypes.sizeof(at.Strides)}, \"strides\");\n"
           f"_Static_assert(sizeof(lr_paged) == {ctypes.sizeof(at.Paged)}, \"paged\");\n"
           f"_Static_assert(sizeof(lr_qk_maps) == {ctypes.sizeof(at.QkMaps)}, \"maps\");\n"
           "int main(void) { return 0; }\n")
    inc = [a for d in ("/usr/local/cuda/include",) if os.path.isdir(d) for a in ("-I", d)]
    r = subprocess.run(["gcc", "-std=c11", "-fsyntax-only", "-x", "c", "-I", os.path.join(ROOT, "include"),
                        *inc, "-"], input=src, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


_CHILD = r"""
import ctypes, sys
sys.path.insert(0, sys.argv[1])
import gated_delta_rule_fwd_gb300 as lr
from gated_delta_rule_fwd_gb300.attention import Strides, Paged, QkMaps
L = lr.lib()
A = [0x10000000 * (i + 1) for i in range(14)]   # distinct, aligned, never dereferenced
P = lambda a: None if a is None else ctypes.c_void_p(a)
def contig(H, T, d): return (H * T * d, T * d, d)
def rope(**kw):
    a = dict(q=A[0], k=A[1], pos=A[2], qo=A[3], ko=A[4], v=A[5], ck=A[6], cv=A[7], tab=A[8],
             qw=A[9], kw=A[10], f=A[11], flags=1, eps=1e-6, rot=32, pages=4, page=16, most=4,
             B=2, T=5, Hq=4, Hk=2, d=64, dt=1, cache=True, maps=True, qs=None, ks=None, vs=None)
    a.update(kw)
    S = lambda s, H: Strides(*(s or contig(H, max(a['T'], 1), a['d'])))
    m = QkMaps(a['flags'], a['qw'], a['kw'], a['eps'], a['rot'], a['f'])
    c = Paged(a['ck'], a['cv'], a['tab'], a['pages'], a['page'], a['most'])
    return L.lr_qk_norm_rope(P(a['q']), S(a['qs'], a['Hq']), P(a['k']), S(a['ks'], a['Hk']), P(a['pos']),
                             ctypes.byref(m) if a['maps'] else None, P(a['qo']), P(a['ko']), P(a['v']),
                             S(a['vs'], a['Hk']), ctypes.byref(c) if a['cache'] else None,
                             a['B'], a['T'], a['Hq'], a['Hk'], a['d'], a['dt'], None)
def win(**kw):
    a = dict(q=A[0], k=A[1], v=A[2], ql=A[3], kl=A[4], o=A[5], B=2, Hq=4, Hk=2, Tq=5, Tk=9, d=64,
             w=4, s=1, scale=0.5, dt=1, qs=None, ks=None, vs=None, os=None)
    a.update(kw)
    S = lambda s, H, T: Strides(*(s or contig(H, max(T, 1), a['d'])))
    return L.lr_fwd_window(P(a['q']), S(a['qs'], a['Hq'], a['Tq']), P(a['k']), S(a['ks'], a['Hk'], a['Tk']),
                           P(a['v']), S(a['vs'], a['Hk'], a['Tk']), P(a['ql']), P(a['kl']), P(a['o']),
                           S(a['os'], a['Hq'], a['Tq']), a['B'], a['Hq'], a['Hk'], a['Tq'], a['Tk'], a['d'],
                           a['w'], a['s'], a['scale'], a['dt'], None)
def step(**kw):
    a = dict(q=A[0], ck=A[1], cv=A[2], tab=A[3], lens=A[4], o=A[5], ws=A[6], wsb=1 << 26, N=3, Hq=4,
             Hk=2, d=64, most_len=9000, w=1 << 30, s=0, scale=0.5, dt=1, pages=9, page=16, most=600, cache=True)
    a.update(kw)
    c = Paged(a['ck'], a['cv'], a['tab'], a['pages'], a['page'], a['most'])
    return L.lr_step_paged(P(a['q']), ctypes.byref(c) if a['cache'] else None, P(a['lens']), P(a['o']), a['N'],
                           a['Hq'], a['Hk'], a['d'], a['most_len'], a['w'], a['s'], a['scale'], a['dt'],
                           P(a['ws']), a['wsb'], None)
wsz = lambda *a: L.lr_step_paged_workspace_size(*a)
need = wsz(3, 4, 2, 64, 9000, 1 << 30, 0, 1)
inf, nan = float('inf'), float('nan')
cases = [
    ("rope-ok", rope(), 7), ("rope-nocache-ok", rope(cache=False, v=None), 7),
    ("rope-T0", rope(T=0, q=None), 0), ("rope-dtype", rope(dt=2), 3), ("rope-d48", rope(d=48), 6),
    ("rope-d0", rope(d=0), 2), ("rope-B0", rope(B=0), 2), ("rope-Tneg", rope(T=-1), 2),
    ("rope-Hk0", rope(Hk=0), 2), ("rope-huge", rope(B=1 << 20, T=1 << 20), 2),
    ("rope-flag", rope(flags=4), 12), ("rope-eps", rope(eps=-1.0), 12), ("rope-eps-nan", rope(eps=nan), 12),
    ("rope-eps-unused", rope(flags=0, eps=nan), 7),
    ("rope-rot-odd", rope(rot=24), 6), ("rope-rot-wide", rope(rot=80), 6), ("rope-rot-neg", rope(rot=-16), 6),
    ("rope-null-maps", rope(maps=False), 1), ("rope-null-freq", rope(f=None), 1),
    ("rope-null-freq-ok", rope(f=None, rot=0), 7),
    ("rope-null-q", rope(q=None), 1), ("rope-null-qo", rope(qo=None), 1), ("rope-null-v", rope(v=None), 1),
    ("rope-null-ko-ok", rope(ko=None), 7), ("rope-null-ko", rope(ko=None, cache=False), 1),
    ("rope-null-table", rope(tab=None), 1), ("rope-page", rope(page=24), 6), ("rope-page8", rope(page=8), 6),
    ("rope-pages0", rope(pages=0), 2), ("rope-most-wide", rope(most=1 << 27), 2),
    ("rope-align-q", rope(q=A[0] + 8), 4), ("rope-align-pos", rope(pos=A[2] + 2), 4),
    ("rope-align-pos-ok", rope(pos=A[2] + 4), 7), ("rope-align-w", rope(qw=A[9] + 4), 4),
    ("rope-stride-neg", rope(qs=(1280, -320, 64)), 2), ("rope-stride-0", rope(ks=(640, 0, 64)), 2),
    ("rope-stride-odd", rope(qs=(1280, 320, 68)), 4),
    ("rope-stride-unused", rope(B=1, qs=(-5, 320, 64)), 7),
    ("rope-alias-qo-q", rope(qo=A[0]), 8), ("rope-alias-ko-qo", rope(ko=A[3] + 64), 8),
    ("rope-alias-cache-k", rope(ck=A[1]), 8), ("rope-alias-pools", rope(cv=A[6] + 128), 8),
    ("rope-alias-qo-pos", rope(qo=A[2]), 8), ("rope-alias-qo-w", rope(qo=A[9]), 8),
    ("rope-alias-w-unused", rope(qo=A[9], flags=0), 7),
    ("win-ok", win(), 7), ("win-Tq0", win(Tq=0, q=None), 0), ("win-Tk0-ok", win(Tk=0, k=None, v=None), 7),
    ("win-dtype", win(dt=-1), 3), ("win-d256", win(d=256), 6), ("win-heads", win(Hq=5), 2),
    ("win-Hk0", win(Hk=0), 2), ("win-window0", win(w=0), 2), ("win-sinks", win(s=-1), 2),
    ("win-scale", win(scale=inf), 2), ("win-scale-nan", win(scale=nan), 2), ("win-B0", win(B=0), 2),
    ("win-Tneg", win(Tk=-1), 2), ("win-huge", win(Tq=1 << 30, B=1 << 10), 2),
    ("win-nullk", win(k=None), 1), ("win-nullo", win(o=None), 1), ("win-null-len-ok", win(ql=None, kl=None), 7),
    ("win-align", win(v=A[2] + 4), 4), ("win-align-len", win(kl=A[4] + 1), 4),
    ("win-o-rows-overlap", win(os=(1280, 320, 32)), 8), ("win-o-heads-first-ok", win(os=(1280, 64, 256)), 7),
    ("win-alias-q", win(o=A[0] + 1024), 8), ("win-alias-len", win(o=A[3] - 1024), 8),
    ("win-stride-k0", win(ks=(1152, 0, 64)), 2), ("win-stride-odd", win(vs=(1152, 576, 60)), 4),
    ("step-ok", step(), 7), ("step-dtype", step(dt=9), 3), ("step-d16", step(d=16), 6), ("step-N0", step(N=0), 2),
    ("step-heads", step(Hq=3), 2), ("step-window", step(w=0), 2), ("step-sinks", step(s=-2), 2),
    ("step-scale", step(scale=nan), 2), ("step-maxlen0", step(most_len=0), 2),
    ("step-maxlen-table", step(most_len=16 * 600 + 1), 2), ("step-null", step(lens=None), 1),
    ("step-null-cache", step(cache=False), 1), ("step-null-pool", step(cv=None), 1), ("step-page", step(page=512), 6),
    ("step-align", step(o=A[5] + 8), 4), ("step-alias-q", step(o=A[0]), 8), ("step-alias-pool", step(o=A[2] + 64), 8),
    ("step-ws-null", step(ws=None), 10), ("step-ws-short", step(wsb=need - 1), 10),
    ("step-ws-align", step(ws=A[6] + 8), 4), ("step-ws-alias", step(ws=A[5]), 8),
    ("step-many", step(N=1 << 30, Hq=4, Hk=4), 2),
    ("ws-split", int(need > 0), 1), ("ws-one-chunk", wsz(3, 4, 2, 64, 64, 1 << 30, 0, 1), 0),
    ("ws-cluster", wsz(3, 4, 2, 64, 300, 1 << 30, 0, 1), 0),
    ("ws-window", wsz(3, 4, 2, 64, 30000, 60, 4, 1), 0), ("ws-bad", wsz(3, 4, 3, 64, 300, 1, 0, 1), 0),
    ("ws-overflow", int(wsz(1, 1, 1, 128, 1 << 30, 0x7fffffff, 0x7fffffff, 0) > 0), 1),
]
bad = [(n, got, want) for n, got, want in cases if got != want]
print("BAD", bad)
sys.exit(1 if bad else 0)
"""


def test_invalid_arguments_rejected_before_launch(lib):
    """In a child without a GPU: a call that passes validation then fails at
    its launch (LR_ERR_CUDA, 7)."""
    env = dict(os.environ, CUDA_VISIBLE_DEVICES="")
    r = subprocess.run([sys.executable, "-c", _CHILD, ROOT], env=env, capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout + r.stderr


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


def test_binding_accepts_what_it_should(lr):
    """The refusals below are the changes' own: unchanged, the calls get as far as the library."""
    f = torch.zeros(32, dtype=torch.float64)
    with pytest.raises(AssertionError, match="lr_fwd_window"):
        lr.lr_fwd_window(_t(1, 4, 9, 64), _t(1, 2, 9, 64), _t(1, 2, 9, 64))
    with pytest.raises(AssertionError, match="lr_step_paged"):
        lr.lr_step_paged(_t(3, 4, 64), _t(5, 2, 16, 64), _t(5, 2, 16, 64), torch.zeros(3, 4, dtype=torch.int32),
                         torch.zeros(3, dtype=torch.int32), max_len=60)
    with pytest.raises(AssertionError, match="lr_qk_norm_rope"):
        lr.lr_qk_norm_rope(_t(2, 4, 9, 64), _t(2, 2, 9, 64), torch.zeros(2, 9, dtype=torch.int32), inv_freq=f,
                           v=_t(2, 2, 9, 64), k_cache=_t(5, 2, 16, 64), v_cache=_t(5, 2, 16, 64),
                           table=torch.zeros(2, 4, dtype=torch.int32), write_k=False)


def _t(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype)


@pytest.mark.parametrize("change", [
    dict(k=_t(1, 2, 9, 32)), dict(k=_t(1, 2, 9, 64, dtype=torch.float32)), dict(q=_t(2, 9, 64)),
    dict(q=_t(1, 4, 64, 9).transpose(2, 3)), dict(q_len=torch.zeros(1, dtype=torch.int64)),
    dict(k_len=torch.zeros(2, dtype=torch.int32)), dict(o=_t(1, 4, 9, 32)), dict(window=1 << 40),
    dict(v=_t(1, 2, 8, 64)), dict(q=_t(1, 4, 9, 64, dtype=torch.float16))])
def test_window_binding_refuses(lr, change):
    a = dict(q=_t(1, 4, 9, 64), k=_t(1, 2, 9, 64), v=_t(1, 2, 9, 64))
    a.update(change)
    q, k, v = a.pop("q"), a.pop("k"), a.pop("v")
    with pytest.raises((ValueError, TypeError)):
        lr.lr_fwd_window(q, k, v, **a)


@pytest.mark.parametrize("change", [
    dict(q=_t(1, 3, 4, 64)), dict(k_cache=_t(5, 2, 16, 32)), dict(v_cache=_t(5, 2, 16, 64, dtype=torch.float32)),
    dict(v_cache=_t(4, 2, 16, 64)), dict(table=torch.zeros(3, 4, dtype=torch.int64)),
    dict(table=torch.zeros(2, 4, dtype=torch.int32)), dict(table=torch.zeros(4, 3, dtype=torch.int32).T),
    dict(lens=torch.zeros(4, dtype=torch.int32)), dict(lens=None), dict(o=_t(3, 4, 32)), dict(max_len=1 << 33)])
def test_step_binding_refuses(lr, change):
    a = dict(q=_t(3, 4, 64), k_cache=_t(5, 2, 16, 64), v_cache=_t(5, 2, 16, 64),
             table=torch.zeros(3, 4, dtype=torch.int32), lens=torch.zeros(3, dtype=torch.int32))
    a.update(change)
    with pytest.raises((ValueError, TypeError)):
        lr.lr_step_paged(**a)


@pytest.mark.parametrize("change", [
    dict(positions=torch.zeros(2, 9, dtype=torch.int64)), dict(positions=torch.zeros(9, dtype=torch.int32)),
    dict(q_weight=_t(64)), dict(inv_freq=torch.zeros(32)), dict(inv_freq=torch.zeros(4, 8, dtype=torch.float64)),
    dict(k_cache=_t(5, 2, 16, 64)), dict(write_k=False), dict(q_out=_t(2, 4, 8, 64)),
    dict(k_out=_t(2, 2, 9, 64, dtype=torch.float32)), dict(k=_t(1, 2, 9, 64)),
    dict(v=_t(2, 2, 9, 64), k_cache=_t(5, 3, 16, 64), v_cache=_t(5, 3, 16, 64),
         table=torch.zeros(2, 4, dtype=torch.int32)),
    dict(v=_t(2, 2, 9, 64), k_cache=_t(5, 2, 16, 64), v_cache=_t(5, 2, 16, 64),
         table=torch.zeros(2, 4, dtype=torch.int32), write_k=False, k_out=_t(2, 2, 9, 64))])
def test_norm_rope_binding_refuses(lr, change):
    a = dict(q=_t(2, 4, 9, 64), k=_t(2, 2, 9, 64))
    a.update(change)
    q, k = a.pop("q"), a.pop("k")
    with pytest.raises((ValueError, TypeError)):
        lr.lr_qk_norm_rope(q, k, **a)


def test_step_fill_refuses_what_the_step_refuses(lib):
    """The same table of refusals for lr_step_paged_fill; the flags that ask for zeros are known ones."""
    child = _CHILD.replace("L.lr_step_paged(", "L.lr_step_paged_fill(").replace(
        "bad = [", 'cases += [("rope-zero", rope(flags=0x19), 7), ("rope-flag-next", rope(flags=0x20), 12)]\nbad = [')
    assert child.count("lr_step_paged_fill") == 1 and "rope-zero" in child
    env = dict(os.environ, CUDA_VISIBLE_DEVICES="")
    r = subprocess.run([sys.executable, "-c", child, ROOT], env=env, capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout + r.stderr


def test_binding_asks_for_zeros_only_in_outputs_that_it_makes(lr, monkeypatch):
    from gated_delta_rule_fwd_gb300 import attention as at
    calls = []

    class Records:
        def __getattr__(self, name):
            return lambda *a: calls.append((name, a)) or 0
    monkeypatch.setattr(lr, "lib", lambda: Records())
    monkeypatch.setattr(at, "_handle", lambda torch, dev: None)
    monkeypatch.setattr(at, "_step_workspace", lambda *a: 0)
    q, k, pos = _t(2, 4, 9, 64), _t(2, 2, 9, 64), torch.zeros(2, 9, dtype=torch.int32)
    for kw, want in ((dict(), 0x18), (dict(q_out=_t(2, 4, 9, 64)), 0x10), (dict(k_out=_t(2, 2, 9, 64)), 0x8),
                     (dict(q_out=_t(2, 4, 9, 64), k_out=_t(2, 2, 9, 64)), 0)):
        lr.lr_qk_norm_rope(q, k, pos, **kw)
        assert calls[-1][1][5].flags & 0x18 == want
    lr.lr_qk_norm_rope(q, k)   # no padding without positions
    assert calls[-1][1][5].flags & 0x18 == 0
    args = (_t(3, 4, 64), _t(5, 2, 16, 64), _t(5, 2, 16, 64), torch.zeros(3, 4, dtype=torch.int32),
            torch.zeros(3, dtype=torch.int32))
    lr.lr_step_paged(*args)
    assert calls[-1][0] == "lr_step_paged_fill"
    lr.lr_step_paged(*args, o=_t(3, 4, 64))
    assert calls[-1][0] == "lr_step_paged"


def test_norm_rope_takes_any_number_of_heads_that_fits(lib):
    child = _CHILD[:_CHILD.index("cases = [")] + '''
cases = [("many-q", rope(B=1, T=1, Hq=70000, Hk=1, cache=False, v=None, d=32, rot=32), 7),
         ("many-k", rope(B=1, T=1, Hq=3, Hk=40000, cache=False, v=None, d=32, rot=32), 7),
         ("too-many", rope(B=1, T=1, Hq=(1 << 30) + 1, Hk=1, cache=False, v=None, d=32, rot=32), 2)]
''' + _CHILD[_CHILD.index("bad = ["):]
    env = dict(os.environ, CUDA_VISIBLE_DEVICES="")
    r = subprocess.run([sys.executable, "-c", child, ROOT], env=env, capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout + r.stderr
