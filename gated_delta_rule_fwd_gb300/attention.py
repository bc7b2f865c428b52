"""Softmax-attention operators of liblr: binding of ``include/lr_attn.h``.

    lr_qk_norm_rope(q, k, positions, ...) -> (q_out, k_out)
        RMS norm of every query and key head and the position rotation in one
        pass, with an optional write of keys and values into a paged cache
    lr_qk_norm_rope_axes(q, k, positions, axis, places, ...) -> (q_out, k_out)
        the same with positions of several axes
    lr_fwd_window(q, k, v, window=..., sinks=...) -> o
        causal attention over whole sequences with a sliding window and sinks
    lr_step_paged(q, k_cache, v_cache, table, lens, ...) -> o
        the same attention for one new token per sequence over the cache
    lr_step_paged_prefix(q, k_cache, v_cache, prefix, prefix_len, table, lens, ...) -> o
        that step for a batch that shares a long prefix
    lr_fwd_diff(q, k, v, lam, ...) -> o
        differential attention over whole sequences
    lr_step_paged_diff(q, k_cache, v_cache, table, lens, lam, ...) -> o
        the same for one new token per sequence over the cache

Like the rest of the package this only marshals arguments; the functions are
offered by the package itself.  Tensors may be on any device: the calls run
there, on its current stream unless one is given.
"""
from __future__ import annotations

import ctypes
import functools

NO_WINDOW = (1 << 31) - 1   # a window that hides nothing
QK_NORM = 0x1
QK_INTERLEAVED = 0x2
QK_ZERO_Q, QK_ZERO_K = 0x8, 0x10
DIFF_NORM, DIFF_FILL = 0x1, 0x2
STEP_FILL = 0x1
MAX_AXES = 16               # LR_MAX_AXES
ATTN_SYMBOLS = ("lr_qk_norm_rope", "lr_qk_norm_rope_axes", "lr_fwd_window", "lr_step_paged", "lr_step_paged_fill",
                "lr_step_paged_workspace_size", "lr_fwd_diff", "lr_fwd_diff_workspace_size",
                "lr_step_paged_diff", "lr_step_paged_diff_workspace_size", "lr_step_paged_prefix",
                "lr_step_paged_prefix_workspace_size")


class Strides(ctypes.Structure):
    """lr_strides (include/lr_attn.h)."""
    _fields_ = [("b", ctypes.c_longlong), ("h", ctypes.c_longlong), ("t", ctypes.c_longlong)]


class Paged(ctypes.Structure):
    """lr_paged (include/lr_attn.h)."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("table", ctypes.c_void_p),
                ("num_pages", ctypes.c_int), ("page", ctypes.c_int), ("max_pages", ctypes.c_int)]


class QkMaps(ctypes.Structure):
    """lr_qk_maps (include/lr_attn.h)."""
    _fields_ = [("flags", ctypes.c_uint), ("q_weight", ctypes.c_void_p),
                ("k_weight", ctypes.c_void_p), ("eps", ctypes.c_float), ("rot", ctypes.c_int),
                ("inv_freq", ctypes.c_void_p)]


class DiffMaps(ctypes.Structure):
    """lr_diff_maps (include/lr_attn.h)."""
    _fields_ = [("flags", ctypes.c_uint), ("lam", ctypes.c_void_p), ("weight", ctypes.c_void_p),
                ("eps", ctypes.c_float)]


_NO_STRIDES = Strides(0, 0, 0)


def declare(L):
    """Argument types of the attention entry points on a loaded library."""
    vp, i, f, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    L.lr_qk_norm_rope.restype = i
    L.lr_qk_norm_rope.argtypes = [vp, Strides, vp, Strides, vp, ctypes.POINTER(QkMaps), vp, vp, vp,
                                  Strides, ctypes.POINTER(Paged)] + [i] * 6 + [vp]
    L.lr_qk_norm_rope_axes.restype = i
    L.lr_qk_norm_rope_axes.argtypes = [vp, Strides, vp, Strides, vp, vp, i, vp, ctypes.POINTER(QkMaps),
                                       vp, vp, vp, Strides, ctypes.POINTER(Paged)] + [i] * 6 + [vp]
    L.lr_fwd_window.restype = i
    L.lr_fwd_window.argtypes = ([vp, Strides] * 3 + [vp, vp, vp, Strides] + [i] * 8 + [f, i, vp])
    L.lr_fwd_diff.restype = i
    L.lr_fwd_diff.argtypes = ([vp, Strides] * 3 + [vp, vp, ctypes.POINTER(DiffMaps), vp, Strides] + [i] * 8 +
                              [f, i, vp, sz, vp])
    L.lr_fwd_diff_workspace_size.restype = sz
    L.lr_fwd_diff_workspace_size.argtypes = [i] * 7
    L.lr_step_paged_diff.restype = i
    L.lr_step_paged_diff.argtypes = ([vp, ctypes.POINTER(Paged), vp, ctypes.POINTER(DiffMaps), vp] + [i] * 7 +
                                     [f, i, vp, sz, vp])
    L.lr_step_paged_diff_workspace_size.restype = sz
    L.lr_step_paged_diff_workspace_size.argtypes = [i] * 8
    L.lr_step_paged_prefix.restype = i
    L.lr_step_paged_prefix.argtypes = ([vp, ctypes.POINTER(Paged), vp, i, vp, vp] + [i] * 7 +
                                       [f, ctypes.c_uint, i, vp, sz, vp])
    L.lr_step_paged_prefix_workspace_size.restype = sz
    L.lr_step_paged_prefix_workspace_size.argtypes = [i] * 9
    for step in (L.lr_step_paged, L.lr_step_paged_fill):
        step.restype = i
        step.argtypes = ([vp, ctypes.POINTER(Paged), vp, vp] + [i] * 7 + [f, i, vp, sz, vp])
    L.lr_step_paged_workspace_size.restype = sz
    L.lr_step_paged_workspace_size.argtypes = [i] * 8


def _base():
    import gated_delta_rule_fwd_gb300 as base
    return base


# The checks below ask for everything at once and look for what is wrong only
# when something is: these calls run once per layer and token, where the time
# of the binding is the time of the step.

def _want(t, name, shape, dtype, dev):
    """A contiguous tensor of this shape, type and device."""
    if t.dtype is not dtype or t.shape != shape or t.device != dev or not t.is_contiguous():
        _base()._check(t, name, shape, dtype, dev)


def _strided(t, name, shape, dtype, dev):
    """A [B, H, T, d] tensor with contiguous channels; its strides."""
    if t.dtype is not dtype or t.shape != shape or t.device != dev:
        _base()._check(t, name, shape, dtype, dev)
    st = t.stride()
    if st[3] != 1 and shape[3] != 1:
        raise ValueError(f"{name} must have contiguous channels")
    return Strides(st[0], st[1], st[2])


def _paged(torch, k_cache, v_cache, table, rows, d, dtype, dev):
    """Pools [P, Hk, page, d] and a table [rows, max_pages]."""
    pool, most = k_cache.shape, table.shape
    if len(pool) != 4 or pool[3] != d:
        raise ValueError(f"k_cache must have shape (pages, heads, page, {d}), got {tuple(pool)}")
    _want(k_cache, "k_cache", pool, dtype, dev)
    _want(v_cache, "v_cache", pool, dtype, dev)
    if len(most) != 2:
        raise ValueError(f"table must have shape ({rows}, pages of a sequence), got {tuple(most)}")
    _want(table, "table", (rows, most[1]), torch.int32, dev)
    return Paged(k_cache.data_ptr(), v_cache.data_ptr(), table.data_ptr(), pool[0], pool[2], most[1])


def _place(torch, stream, dev):
    """The given stream, or the device's current one, made current: a call
    allocates and launches there, and what it allocates belongs to it."""
    if stream is None:
        return torch.cuda.device(dev)
    if stream.device != dev:
        raise ValueError(f"stream must be on {dev}, got {stream.device}")
    return torch.cuda.stream(stream)


def _handle(torch, dev):
    """The current stream of the device."""
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return raw(dev.index) if raw else torch.cuda.current_stream(dev).cuda_stream


def _int32(x, name):
    x = int(x)
    if not -(1 << 31) <= x < (1 << 31):
        raise ValueError(f"{name} does not fit 32 bits: {x}")
    return x


def lr_qk_norm_rope(q, k, positions=None, *, norm=True, q_weight=None, k_weight=None, eps=1e-6,
                    inv_freq=None, interleaved=False, v=None, k_cache=None, v_cache=None,
                    table=None, write_k=True, q_out=None, k_out=None, stream=None):
    """Norm and rotation of queries and keys (``lr_qk_norm_rope`` in include/lr_attn.h).

    q: [B,Hq,T,d]; k: [B,Hk,T,d] (float32 or bfloat16), any strides with
    contiguous channels, e.g. transposed views of one projection;
    positions: [B,T] int32 (negative: padding, left out) or None for 0..T-1;
    q_weight, k_weight: [d] float32 or None, of the norm; inv_freq: [rot/2] float64 radians
    per position, or None for no rotation; ``interleaved`` rotates channels
    (2i, 2i+1) instead of (i, i + rot/2).  With k_cache, v_cache
    [pages,Hk,page,d], table [B,max_pages] int32 and v [B,Hk,T,d], the keys
    and v are also written at their positions in the cache; then
    ``write_k=False`` leaves out the contiguous keys.  Returns (q_out, k_out)
    [B,H,T,d] contiguous (k_out None without ``write_k``); rows of padding are
    left as they were in outputs that are given, zeros in those made here."""
    import torch
    base = _base()
    dev = q.device
    base._require_cuda(dev)
    if stream is not None or torch.cuda.current_device() != dev.index:
        with _place(torch, stream, dev):
            return lr_qk_norm_rope(q, k, positions, norm=norm, q_weight=q_weight, k_weight=k_weight,
                                   eps=eps, inv_freq=inv_freq, interleaved=interleaved, v=v,
                                   k_cache=k_cache, v_cache=v_cache, table=table, write_k=write_k,
                                   q_out=q_out, k_out=k_out)
    return _norm_rope(torch, base, q, k, positions, None, None, norm, q_weight, k_weight, eps, inv_freq,
                      interleaved, v, k_cache, v_cache, table, write_k, q_out, k_out)


def lr_qk_norm_rope_axes(q, k, positions, axis, places=None, *, norm=True, q_weight=None, k_weight=None,
                         eps=1e-6, inv_freq=None, interleaved=False, v=None, k_cache=None, v_cache=None,
                         table=None, write_k=True, q_out=None, k_out=None, stream=None):
    """Norm and rotation by positions of several axes (``lr_qk_norm_rope_axes`` in
    include/lr_attn.h).

    positions: [axes,B,T] int32, e.g. time, height and width of every token;
    axis: [rot/2] int32, the axis of each frequency's channel pair (in runs or
    in turn, as the model has it); places: [B,T] int32 rows of the tokens in
    their sequence's cache (negative: padding, left out) or None for 0..T-1.
    The other arguments and the results are those of :func:`lr_qk_norm_rope`."""
    import torch
    base = _base()
    dev = q.device
    base._require_cuda(dev)
    if stream is not None or torch.cuda.current_device() != dev.index:
        with _place(torch, stream, dev):
            return lr_qk_norm_rope_axes(q, k, positions, axis, places, norm=norm, q_weight=q_weight,
                                        k_weight=k_weight, eps=eps, inv_freq=inv_freq, interleaved=interleaved,
                                        v=v, k_cache=k_cache, v_cache=v_cache, table=table, write_k=write_k,
                                        q_out=q_out, k_out=k_out)
    if positions is None or axis is None:
        raise ValueError("positions and axis are required")
    return _norm_rope(torch, base, q, k, places, positions, axis, norm, q_weight, k_weight, eps, inv_freq,
                      interleaved, v, k_cache, v_cache, table, write_k, q_out, k_out)


def _norm_rope(torch, base, q, k, places, positions, axis, norm, q_weight, k_weight, eps, inv_freq, interleaved,
               v, k_cache, v_cache, table, write_k, q_out, k_out):
    """Either norm and rotation; without ``axis`` the places are the positions."""
    dev = q.device
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError("q and k must have shape (B, heads, T, d)")
    q_shape, k_shape, dtype = q.shape, k.shape, q.dtype
    B, Hq, T, d = q_shape
    Hk = k_shape[1]
    dt = base._dtype_code(q)
    qs = _strided(q, "q", q_shape, dtype, dev)
    ks = _strided(k, "k", (B, Hk, T, d), dtype, dev)
    if places is not None:
        _want(places, "positions" if axis is None else "places", (B, T), torch.int32, dev)
    if q_weight is not None:
        _want(q_weight, "q_weight", (d,), torch.float32, dev)
    if k_weight is not None:
        _want(k_weight, "k_weight", (d,), torch.float32, dev)
    rot = 0
    if inv_freq is not None:
        rot = 2 * inv_freq.numel()
        _want(inv_freq, "inv_freq", (rot // 2,), torch.float64, dev)
    if axis is not None:
        axes = positions.shape[0] if positions.dim() == 3 else 0
        if not 1 <= axes <= MAX_AXES:
            raise ValueError(f"positions must have shape (1 to {MAX_AXES}, {B}, {T}), got {tuple(positions.shape)}")
        _want(positions, "positions", (axes, B, T), torch.int32, dev)
        _want(axis, "axis", (rot // 2,), torch.int32, dev)
    cache, vs = None, _NO_STRIDES
    if k_cache is not None or v_cache is not None or table is not None or v is not None:
        if k_cache is None or v_cache is None or table is None or v is None:
            raise ValueError("a cache needs v, k_cache, v_cache and table together")
        cache = _paged(torch, k_cache, v_cache, table, B, d, dtype, dev)
        if k_cache.shape[1] != Hk:
            raise ValueError(f"k_cache must have {Hk} heads, got {k_cache.shape[1]}")
        vs = _strided(v, "v", k_shape, dtype, dev)
    elif not write_k:
        raise ValueError("write_k=False needs a cache")
    if q_out is not None:
        _want(q_out, "q_out", q_shape, dtype, dev)
    if k_out is not None:
        if not write_k:
            raise ValueError("k_out given with write_k=False")
        _want(k_out, "k_out", k_shape, dtype, dev)
    flags = (QK_NORM if norm else 0) | (QK_INTERLEAVED if interleaved else 0)
    if places is not None:
        flags |= (QK_ZERO_Q if q_out is None else 0) | (QK_ZERO_K if k_out is None else 0)
    maps = QkMaps(flags,
                  None if q_weight is None else q_weight.data_ptr(),
                  None if k_weight is None else k_weight.data_ptr(), float(eps), rot,
                  None if inv_freq is None else inv_freq.data_ptr())
    if q_out is None:
        q_out = torch.empty(q_shape, dtype=dtype, device=dev)
    if k_out is None and write_k:
        k_out = torch.empty(k_shape, dtype=dtype, device=dev)
    L, turns = base.lib(), ()
    if axis is None:
        name, call = "lr_qk_norm_rope", L.lr_qk_norm_rope
    else:
        name, call = "lr_qk_norm_rope_axes", L.lr_qk_norm_rope_axes
        turns = (positions.data_ptr(), axis.data_ptr(), axes)
    st = call(q.data_ptr(), qs, k.data_ptr(), ks, *turns, None if places is None else places.data_ptr(),
              maps, q_out.data_ptr(), None if k_out is None else k_out.data_ptr(),
              None if v is None else v.data_ptr(), vs, cache, B, T, Hq, Hk, d, dt, _handle(torch, dev))
    if st != 0:
        raise base.LrError(st, name)
    return q_out, k_out


def lr_fwd_window(q, k, v, *, window=None, sinks=0, q_len=None, k_len=None, scale=None, o=None,
                  stream=None):
    """Causal attention with a sliding window and sinks (``lr_fwd_window`` in
    include/lr_attn.h).

    q: [B,Hq,Tq,d]; k, v: [B,Hk,Tk,d] (float32 or bfloat16), any strides with
    contiguous channels; Hq a multiple of Hk.  The queries are the last tokens
    of the keys' sequence.  window: tokens a row sees, itself included (None:
    all before it); sinks: first tokens that stay visible; q_len, k_len: [B]
    int32 lengths of a padded batch or None; scale: default d**-0.5.  ``o``
    may be strided too; rows behind q_len are left as they were (zeros when o
    is made here).  Returns o: [B,Hq,Tq,d]."""
    import torch
    base = _base()
    dev = q.device
    base._require_cuda(dev)
    if stream is not None or torch.cuda.current_device() != dev.index:
        with _place(torch, stream, dev):
            return lr_fwd_window(q, k, v, window=window, sinks=sinks, q_len=q_len, k_len=k_len,
                                 scale=scale, o=o)
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError("q, k and v must have shape (B, heads, T, d)")
    q_shape, dtype = q.shape, q.dtype
    B, Hq, Tq, d = q_shape
    _, Hk, Tk, _ = k.shape
    dt = base._dtype_code(q)
    qs = _strided(q, "q", q_shape, dtype, dev)
    ks = _strided(k, "k", (B, Hk, Tk, d), dtype, dev)
    vs = _strided(v, "v", (B, Hk, Tk, d), dtype, dev)
    if q_len is not None:
        _want(q_len, "q_len", (B,), torch.int32, dev)
    if k_len is not None:
        _want(k_len, "k_len", (B,), torch.int32, dev)
    os_ = None if o is None else _strided(o, "o", q_shape, dtype, dev)
    window = NO_WINDOW if window is None else _int32(window, "window")
    sinks = _int32(sinks, "sinks")
    scale = d ** -0.5 if scale is None else float(scale)
    if o is None:
        o = (torch.empty if q_len is None else torch.zeros)(q_shape, dtype=dtype, device=dev)
        os_ = _strided(o, "o", q_shape, dtype, dev)
    st = base.lib().lr_fwd_window(
        q.data_ptr(), qs, k.data_ptr(), ks, v.data_ptr(), vs,
        None if q_len is None else q_len.data_ptr(), None if k_len is None else k_len.data_ptr(),
        o.data_ptr(), os_, B, Hq, Hk, Tq, Tk, d, window, sinks, scale, dt, _handle(torch, dev))
    if st != 0:
        raise base.LrError(st, "lr_fwd_window")
    return o


def _diff_maps(torch, lam, norm, norm_weight, eps, H, d, dev):
    """lr_diff_maps of H pairs of heads."""
    _want(lam, "lam", (H,), torch.float32, dev)
    if norm_weight is not None:
        if not norm:
            raise ValueError("norm_weight given with norm=False")
        _want(norm_weight, "norm_weight", (2 * d,), torch.float32, dev)
    return DiffMaps(DIFF_NORM if norm else 0, lam.data_ptr(),
                    None if norm_weight is None else norm_weight.data_ptr(), float(eps))


def _scratch(torch, workspace, need, dev):
    """A call's workspace, the given one or one made here: its holder, address and size."""
    if workspace is None:
        if need == 0:
            return None, None, 0
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    elif workspace.device != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be contiguous and on {dev}")
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


@functools.lru_cache(maxsize=1024)
def _diff_workspace(B, H, Hk, Tq, Tk, d, dt):
    """lr_fwd_diff_workspace_size, a function of the sizes alone."""
    return int(_base().lib().lr_fwd_diff_workspace_size(B, H, Hk, Tq, Tk, d, dt))


def diff_workspace_size(B, H, Hk, Tq, Tk, d, dtype) -> int:
    """lr_fwd_diff_workspace_size for these sizes (H and Hk pairs of heads; dtype: torch dtype)."""
    import torch
    base = _base()
    return _diff_workspace(B, H, Hk, Tq, Tk, d, base.F32 if dtype == torch.float32 else base.BF16)


def lr_fwd_diff(q, k, v, lam, *, window=None, sinks=0, q_len=None, k_len=None, scale=None, norm=True,
                norm_weight=None, eps=1e-6, o=None, workspace=None, stream=None):
    """Differential attention over whole sequences (``lr_fwd_diff`` in
    include/lr_attn.h).

    q: [B,2H,Tq,d]; k, v: [B,2Hk,Tk,d] (float32 or bfloat16), any strides with
    contiguous channels; H a multiple of Hk.  Heads 2h and 2h+1 of q and k are
    the two maps of pair h; those of v and o are the halves of its 2d value
    channels.  lam: [H] float32, the second map's factor.  ``norm``: the
    root-mean-square norm of every pair's row, times norm_weight ([2d] float32 or
    None for ones; a factor 1 - lambda_init belongs into it).  window, sinks,
    q_len, k_len, scale and ``o`` as for :func:`lr_fwd_window`.  ``workspace`` is
    a uint8 CUDA tensor of at least ``diff_workspace_size(...)`` bytes, allocated
    here when None.  Returns o: [B,2H,Tq,d]."""
    import torch
    base = _base()
    dev = q.device
    base._require_cuda(dev)
    if stream is not None or torch.cuda.current_device() != dev.index:
        with _place(torch, stream, dev):
            return lr_fwd_diff(q, k, v, lam, window=window, sinks=sinks, q_len=q_len, k_len=k_len, scale=scale,
                               norm=norm, norm_weight=norm_weight, eps=eps, o=o, workspace=workspace)
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError("q, k and v must have shape (B, heads, T, d)")
    q_shape, dtype = q.shape, q.dtype
    B, H2, Tq, d = q_shape
    _, Hk2, Tk, _ = k.shape
    if H2 % 2 or Hk2 % 2:
        raise ValueError(f"heads come in pairs, got {H2} and {Hk2}")
    dt = base._dtype_code(q)
    qs = _strided(q, "q", q_shape, dtype, dev)
    ks = _strided(k, "k", (B, Hk2, Tk, d), dtype, dev)
    vs = _strided(v, "v", (B, Hk2, Tk, d), dtype, dev)
    if q_len is not None:
        _want(q_len, "q_len", (B,), torch.int32, dev)
    if k_len is not None:
        _want(k_len, "k_len", (B,), torch.int32, dev)
    maps = _diff_maps(torch, lam, norm, norm_weight, eps, H2 // 2, d, dev)
    os_ = None if o is None else _strided(o, "o", q_shape, dtype, dev)
    window = NO_WINDOW if window is None else _int32(window, "window")
    sinks = _int32(sinks, "sinks")
    scale = d ** -0.5 if scale is None else float(scale)
    L = base.lib().lr_fwd_diff
    need = 0 if workspace is not None else _diff_workspace(B, H2 // 2, Hk2 // 2, Tq, Tk, d, dt)
    held, ws, ws_bytes = _scratch(torch, workspace, need, dev)
    if o is None:
        o = (torch.empty if q_len is None else torch.zeros)(q_shape, dtype=dtype, device=dev)
        os_ = _strided(o, "o", q_shape, dtype, dev)
    st = L(q.data_ptr(), qs, k.data_ptr(), ks, v.data_ptr(), vs, None if q_len is None else q_len.data_ptr(),
           None if k_len is None else k_len.data_ptr(), maps, o.data_ptr(), os_, B, H2 // 2, Hk2 // 2, Tq, Tk, d,
           window, sinks, scale, dt, ws, ws_bytes, _handle(torch, dev))
    if st != 0:
        raise base.LrError(st, "lr_fwd_diff")
    return o


@functools.lru_cache(maxsize=1024)
def _step_workspace(N, Hq, Hk, d, max_len, window, sinks, dt):
    """lr_step_paged_workspace_size, a function of the sizes alone."""
    return int(_base().lib().lr_step_paged_workspace_size(N, Hq, Hk, d, max_len, window, sinks, dt))


def step_paged_workspace_size(N, Hq, Hk, d, max_len, dtype, window=None, sinks=0) -> int:
    """lr_step_paged_workspace_size for these sizes (dtype: torch dtype)."""
    import torch
    base = _base()
    dt = base.F32 if dtype == torch.float32 else base.BF16
    window = NO_WINDOW if window is None else _int32(window, "window")
    return _step_workspace(N, Hq, Hk, d, _int32(max_len, "max_len"), window,
                           _int32(sinks, "sinks"), dt)


def lr_step_paged(q, k_cache, v_cache, table, lens, *, max_len=None, window=None, sinks=0,
                  scale=None, o=None, workspace=None, stream=None):
    """Attention of one new token per sequence over the paged cache
    (``lr_step_paged`` in include/lr_attn.h).

    q: [N,Hq,d]; k_cache, v_cache: [pages,Hk,page,d]; table: [N,max_pages]
    int32; lens: [N] int32 tokens in the cache, this one included (0: a row of
    zeros, negative: an unused slot, whose row is left as it was in an ``o``
    that is given, zeros in one made here); max_len: bound on lens
    (default: what the table can hold; a tight one is faster); window, sinks,
    scale as for :func:`lr_fwd_window`.  ``workspace`` is a uint8 CUDA tensor
    of at least ``step_paged_workspace_size(...)`` bytes, allocated here when
    None.  Returns o: [N,Hq,d]."""
    import torch
    base = _base()
    dev = q.device
    base._require_cuda(dev)
    if stream is not None or torch.cuda.current_device() != dev.index:
        with _place(torch, stream, dev):
            return lr_step_paged(q, k_cache, v_cache, table, lens, max_len=max_len, window=window,
                                 sinks=sinks, scale=scale, o=o, workspace=workspace)
    if q.dim() != 3:
        raise ValueError("q must have shape (N, heads, d)")
    q_shape, dtype = q.shape, q.dtype
    N, Hq, d = q_shape
    dt = base._dtype_code(q)
    _want(q, "q", q_shape, dtype, dev)
    cache = _paged(torch, k_cache, v_cache, table, N, d, dtype, dev)
    Hk = k_cache.shape[1]
    if lens is None:
        raise ValueError("lens is required")
    _want(lens, "lens", (N,), torch.int32, dev)
    if o is not None:
        _want(o, "o", q_shape, dtype, dev)
    max_len = cache.page * cache.max_pages if max_len is None else _int32(max_len, "max_len")
    window = NO_WINDOW if window is None else _int32(window, "window")
    sinks = _int32(sinks, "sinks")
    scale = d ** -0.5 if scale is None else float(scale)
    need = 0
    if workspace is None:
        need = _step_workspace(N, Hq, Hk, d, max_len, window, sinks, dt)
    elif workspace.device != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be contiguous and on {dev}")
    L = base.lib()
    step = L.lr_step_paged
    if o is None:
        o = torch.empty(q_shape, dtype=dtype, device=dev)
        step = L.lr_step_paged_fill
    if need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    ws, ws_bytes = ((None, 0) if workspace is None else
                    (workspace.data_ptr(), workspace.numel() * workspace.element_size()))
    st = step(q.data_ptr(), cache, lens.data_ptr(), o.data_ptr(), N, Hq, Hk, d, max_len, window,
              sinks, scale, dt, ws, ws_bytes, _handle(torch, dev))
    if st != 0:
        raise base.LrError(st, "lr_step_paged")
    return o


@functools.lru_cache(maxsize=1024)
def _step_diff_workspace(N, H, Hk, d, max_len, window, sinks, dt):
    """lr_step_paged_diff_workspace_size, a function of the sizes alone."""
    return int(_base().lib().lr_step_paged_diff_workspace_size(N, H, Hk, d, max_len, window, sinks, dt))


def step_paged_diff_workspace_size(N, H, Hk, d, max_len, dtype, window=None, sinks=0) -> int:
    """lr_step_paged_diff_workspace_size for these sizes (H and Hk pairs of heads; dtype: torch dtype)."""
    import torch
    base = _base()
    dt = base.F32 if dtype == torch.float32 else base.BF16
    window = NO_WINDOW if window is None else _int32(window, "window")
    return _step_diff_workspace(N, H, Hk, d, _int32(max_len, "max_len"), window, _int32(sinks, "sinks"), dt)


def lr_step_paged_diff(q, k_cache, v_cache, table, lens, lam, *, max_len=None, window=None, sinks=0, scale=None,
                       norm=True, norm_weight=None, eps=1e-6, o=None, workspace=None, stream=None):
    """Differential attention of one new token per sequence over the paged cache
    (``lr_step_paged_diff`` in include/lr_attn.h).

    q: [N,2H,d]; k_cache, v_cache: [pages,2Hk,page,d], heads in pairs as for
    :func:`lr_fwd_diff`; lam, norm, norm_weight, eps as there; table, lens,
    max_len, window, sinks, scale, ``o`` as for :func:`lr_step_paged`.
    ``workspace`` is a uint8 CUDA tensor of at least
    ``step_paged_diff_workspace_size(...)`` bytes, allocated here when None.
    Returns o: [N,2H,d]."""
    import torch
    base = _base()
    dev = q.device
    base._require_cuda(dev)
    if stream is not None or torch.cuda.current_device() != dev.index:
        with _place(torch, stream, dev):
            return lr_step_paged_diff(q, k_cache, v_cache, table, lens, lam, max_len=max_len, window=window,
                                      sinks=sinks, scale=scale, norm=norm, norm_weight=norm_weight, eps=eps, o=o,
                                      workspace=workspace)
    if q.dim() != 3:
        raise ValueError("q must have shape (N, heads, d)")
    q_shape, dtype = q.shape, q.dtype
    N, H2, d = q_shape
    dt = base._dtype_code(q)
    _want(q, "q", q_shape, dtype, dev)
    cache = _paged(torch, k_cache, v_cache, table, N, d, dtype, dev)
    Hk2 = k_cache.shape[1]
    if H2 % 2 or Hk2 % 2:
        raise ValueError(f"heads come in pairs, got {H2} and {Hk2}")
    if lens is None:
        raise ValueError("lens is required")
    _want(lens, "lens", (N,), torch.int32, dev)
    maps = _diff_maps(torch, lam, norm, norm_weight, eps, H2 // 2, d, dev)
    if o is not None:
        _want(o, "o", q_shape, dtype, dev)
    max_len = cache.page * cache.max_pages if max_len is None else _int32(max_len, "max_len")
    window = NO_WINDOW if window is None else _int32(window, "window")
    sinks = _int32(sinks, "sinks")
    scale = d ** -0.5 if scale is None else float(scale)
    step = base.lib().lr_step_paged_diff
    need = 0
    if workspace is None:
        need = _step_diff_workspace(N, H2 // 2, Hk2 // 2, d, max_len, window, sinks, dt)
    held, ws, ws_bytes = _scratch(torch, workspace, need, dev)
    if o is None:
        o = torch.empty(q_shape, dtype=dtype, device=dev)
        maps.flags |= DIFF_FILL
    st = step(q.data_ptr(), cache, lens.data_ptr(), maps, o.data_ptr(), N, H2 // 2, Hk2 // 2, d, max_len, window,
              sinks, scale, dt, ws, ws_bytes, _handle(torch, dev))
    if st != 0:
        raise base.LrError(st, "lr_step_paged_diff")
    return o


@functools.lru_cache(maxsize=1024)
def _step_prefix_workspace(N, Hq, Hk, d, prefix_len, max_len, window, sinks, dt):
    """lr_step_paged_prefix_workspace_size, a function of the sizes alone."""
    return int(_base().lib().lr_step_paged_prefix_workspace_size(N, Hq, Hk, d, prefix_len, max_len, window, sinks, dt))


def step_paged_prefix_workspace_size(N, Hq, Hk, d, prefix_len, max_len, dtype, window=None, sinks=0) -> int:
    """lr_step_paged_prefix_workspace_size for these sizes (dtype: torch dtype)."""
    import torch
    base = _base()
    dt = base.F32 if dtype == torch.float32 else base.BF16
    window = NO_WINDOW if window is None else _int32(window, "window")
    return _step_prefix_workspace(N, Hq, Hk, d, _int32(prefix_len, "prefix_len"), _int32(max_len, "max_len"), window,
                                  _int32(sinks, "sinks"), dt)


def lr_step_paged_prefix(q, k_cache, v_cache, prefix, prefix_len, table, lens, *, max_len=None, window=None, sinks=0,
                         scale=None, o=None, workspace=None, stream=None):
    """:func:`lr_step_paged` for sequences that begin with the same tokens
    (``lr_step_paged_prefix`` in include/lr_attn.h).

    prefix: [pages] int32 pages of the shared prefix, in the same pools;
    prefix_len: its tokens (an int).  table and lens are of each sequence's own
    tokens behind it (lens 0: the row of the prefix's last token).  window and
    sinks count in positions of the whole sequence; q, k_cache, v_cache, max_len,
    scale, ``o`` as for :func:`lr_step_paged`.  ``workspace`` is a uint8 CUDA
    tensor of at least ``step_paged_prefix_workspace_size(...)`` bytes, allocated
    here when None.  Returns o: [N,Hq,d]."""
    import torch
    base = _base()
    dev = q.device
    base._require_cuda(dev)
    if stream is not None or torch.cuda.current_device() != dev.index:
        with _place(torch, stream, dev):
            return lr_step_paged_prefix(q, k_cache, v_cache, prefix, prefix_len, table, lens, max_len=max_len,
                                        window=window, sinks=sinks, scale=scale, o=o, workspace=workspace)
    if q.dim() != 3:
        raise ValueError("q must have shape (N, heads, d)")
    q_shape, dtype = q.shape, q.dtype
    N, Hq, d = q_shape
    dt = base._dtype_code(q)
    _want(q, "q", q_shape, dtype, dev)
    cache = _paged(torch, k_cache, v_cache, table, N, d, dtype, dev)
    Hk = k_cache.shape[1]
    prefix_len = _int32(prefix_len, "prefix_len")
    if prefix is None or lens is None:
        raise ValueError("prefix and lens are required")
    if prefix.dim() != 1 or prefix.shape[0] * cache.page < prefix_len:
        raise ValueError(f"prefix must have shape (pages,) with room for {prefix_len} tokens, got {tuple(prefix.shape)}")
    _want(prefix, "prefix", prefix.shape, torch.int32, dev)
    _want(lens, "lens", (N,), torch.int32, dev)
    if o is not None:
        _want(o, "o", q_shape, dtype, dev)
    max_len = cache.page * cache.max_pages if max_len is None else _int32(max_len, "max_len")
    window = NO_WINDOW if window is None else _int32(window, "window")
    sinks = _int32(sinks, "sinks")
    scale = d ** -0.5 if scale is None else float(scale)
    step = base.lib().lr_step_paged_prefix
    need = 0
    if workspace is None:
        need = _step_prefix_workspace(N, Hq, Hk, d, prefix_len, max_len, window, sinks, dt)
    held, ws, ws_bytes = _scratch(torch, workspace, need, dev)
    flags = 0
    if o is None:
        o = torch.empty(q_shape, dtype=dtype, device=dev)
        flags = STEP_FILL
    st = step(q.data_ptr(), cache, prefix.data_ptr(), prefix_len, lens.data_ptr(), o.data_ptr(), N, Hq, Hk, d, max_len,
              window, sinks, scale, flags, dt, ws, ws_bytes, _handle(torch, dev))
    if st != 0:
        raise base.LrError(st, "lr_step_paged_prefix")
    return o
