"""Cached attention: a paged key-value cache with its append, decode, page
choice and sparse attention (the C ABI of include/tiered_attn_cache.h).

Argument marshalling only, as in ``binding``: the operators run in the
library's CUDA kernels, the caller owns every buffer.  A call goes through
``_cache_call`` (csrc/ta_cache_py.cpp), which checks and marshals in C++; what
it refuses is checked again here, for the reason.  Where that module could not
be built, all calls are checked and marshalled here (a warning says so once).
Strides come from the tensors of each call, sizes from the parameters::

    p = pav.make_cache_params(n_pages=P, page_size=64, H=32, Hkv=8, d=128, S=S, T=T,
                              max_pages=W, n_select=16, rot_dim=128)
    ws = pav.alloc_cache_workspace(p, "cuda")
    cache = pav.make_cache(p, "cuda")
    pav.cache_append(p, cache, K, V, table, lens, ws, cu=cu, cos=cos, sin=sin, Q=Q, Q_out=Q)
    pav.cache_select(p, cache, Q, table, lens, ws, sel, cu=cu)
    pav.cache_sparse(p, cache, Q, sel, table, lens, ws, O, cu=cu)

A row sees the keys at positions up to its own, also among the new tokens of a
step: the tokens of one latent frame do not see the ones behind them.  Where they
should, append the frame and attend with a sequence for each row: no ``cu``,
``lens`` the frame's end in every entry, the sequence's table row repeated.
"""

from __future__ import annotations

import ctypes
import warnings
from typing import Optional

import torch

from . import binding as _b
from .binding import TieredAttnError, _check

TA_ERR_BAD_INDEX = -6
TA_CACHE_BF16, TA_CACHE_FP8 = 0, 1

_i32, _i64, _vp = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p


class ta_cache_params(ctypes.Structure):
    _fields_ = [(n, _i32) for n in (
        "n_pages", "page_size", "H", "Hkv", "d", "format", "S", "T", "max_pages", "n_select",
        "n_first", "n_recent", "rot_dim", "rot_interleaved", "rot_rows")] + [
        ("softmax_scale", ctypes.c_float)] + [(n, _i64) for n in (
            "stride_page", "stride_head", "stride_slot", "stride_table", "stride_k_t",
            "stride_k_h", "stride_v_t", "stride_v_h", "stride_q_t", "stride_q_h", "stride_o_t",
            "stride_o_h")]


class ta_cache(ctypes.Structure):
    _fields_ = [(n, _vp) for n in ("k", "v", "k_scale", "v_scale", "k_mean")]


class _CacheView(ctypes.Structure):
    """What ``_cache_call`` reads of a PagedCache (CacheView there)."""
    _fields_ = [("c", ta_cache), ("stride", _i64 * 3), ("shape", _i64 * 4), ("format", _i32),
                ("device", _i32), ("has_mean", _i32), ("pad", _i32)]


_P = ctypes.POINTER(ta_cache_params)
_C = ctypes.POINTER(ta_cache)
_SIGS = {
    "tiered_attn_cache_workspace_bytes": (ctypes.c_size_t, [_P]),
    "tiered_attn_cache_init": (ctypes.c_int, [_vp, ctypes.c_size_t, _vp]),
    "tiered_attn_cache_append": (ctypes.c_int, [_P, _C] + [_vp] * 11 + [ctypes.c_size_t, _vp]),
    "tiered_attn_cache_decode": (ctypes.c_int, [_P, _C] + [_vp] * 6 + [ctypes.c_size_t, _vp]),
    "tiered_attn_cache_select": (ctypes.c_int, [_P, _C] + [_vp] * 6 + [ctypes.c_size_t, _vp]),
    "tiered_attn_cache_sparse": (ctypes.c_int, [_P, _C] + [_vp] * 8 + [ctypes.c_size_t, _vp]),
}
_fns = {}


def _fn(name):
    f = _fns.get(name)
    if f is None:
        f = getattr(_b.lib(), name)
        f.restype, f.argtypes = _SIGS[name]
        _fns[name] = f
    return f


_call = None


class _NoNative:
    """In place of a C++ entry that is not there: refuses every call."""

    @staticmethod
    def append(*args):
        return None

    decode = select = sparse = append


def _native():
    """The C++ entry, bound to the library on first use."""
    global _call
    if _call is None:
        try:
            from . import _cache_call as m
        except ImportError as e:
            _b.lib()                     # (a missing library raises)
            warnings.warn(f"_cache_call.so is missing or does not load ({e}): cached attention is called "
                          "through ctypes, some 10 us a call slower; `python -m "
                          "precision_attention_video_b200.build` builds it", RuntimeWarning, stacklevel=3)
            _call = _NoNative
            return _call
        m.init(*(ctypes.cast(_fn("tiered_attn_cache_" + n), _vp).value
                 for n in ("append", "decode", "select", "sparse")))
        _call = m
    return _call


def make_cache_params(*, n_pages: int, page_size: int, H: int, Hkv: int, d: int, S: int, T: int,
                      max_pages: int, format: int = TA_CACHE_BF16, n_select: int = 0,
                      n_first: int = 1, n_recent: int = 1, rot_dim: int = 0,
                      rot_interleaved: int = 0, softmax_scale: float = 0.0) -> ta_cache_params:
    """Sizes of a cache and of a step: S sequences with T new tokens in all
    (the buffers' rows), at most max_pages pages each.  Rows attend causally,
    among the new tokens too."""
    p = ta_cache_params()
    p.n_pages, p.page_size, p.H, p.Hkv, p.d, p.format = n_pages, page_size, H, Hkv, d, format
    p.S, p.T, p.max_pages = S, T, max_pages
    p.n_select, p.n_first, p.n_recent = n_select, n_first, n_recent
    p.rot_dim, p.rot_interleaved, p.softmax_scale = rot_dim, rot_interleaved, softmax_scale
    return p


class PagedCache:
    """The cache's tensors, each on one CUDA device: ``k`` and ``v`` bf16 or
    float8_e4m3fn [n_pages, Hkv, page_size, d] (any order of the outer three
    dimensions in memory), ``k_scale`` and ``v_scale`` f32 [n_pages, Hkv,
    page_size] for FP8, ``k_mean`` f32 [n_pages, Hkv, d] where pages are
    chosen.  ``k`` and ``v`` may be None for a cache that is only chosen from.
    Calls read the tensors' places from here, so they cannot be exchanged for
    others (nor may their memory be: ``set_``, ``resize_``); make a new
    PagedCache instead."""

    __slots__ = ("k", "v", "k_scale", "v_scale", "k_mean", "_view", "_strides", "_shape", "_fmt",
                 "_dev")

    def __init__(self, k, v, k_scale=None, v_scale=None, k_mean=None):
        some = k if k is not None else k_mean
        if some is None:
            raise ValueError("PagedCache: neither keys nor means")
        self._dev = some.get_device()
        if k is None:
            self._fmt, self._shape, self._strides = None, None, (0, 0, 0)
        else:
            if k.dtype not in (torch.bfloat16, torch.float8_e4m3fn):
                raise TypeError(f"k: expected torch.bfloat16 or torch.float8_e4m3fn, got {k.dtype}")
            if not isinstance(v, torch.Tensor) or v.dtype != k.dtype:
                raise TypeError("v: expected a tensor of k's type")
            if k.dim() != 4 or v.shape != k.shape or v.stride() != k.stride() or k.stride(3) != 1:
                raise ValueError("k, v: expected [n_pages, Hkv, page_size, d] with equal strides, "
                                 "d contiguous")
            self._fmt = TA_CACHE_FP8 if k.dtype == torch.float8_e4m3fn else TA_CACHE_BF16
            self._shape, self._strides = tuple(k.shape), k.stride()[:3]
            if self._fmt == TA_CACHE_FP8:
                for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
                    _plain(name, t, torch.float32, self._shape[:3], self._dev)
        if k_mean is not None:
            if k_mean.dim() != 3:
                raise ValueError("k_mean: expected [n_pages, Hkv, d]")
            want = tuple(k_mean.shape) if k is None else (*self._shape[:2], self._shape[3])
            _plain("k_mean", k_mean, torch.float32, want, self._dev)
        for name, t in (("k", k), ("v", v)):
            if t is not None and t.get_device() != self._dev:
                raise ValueError(f"{name}: not on the cache's device")
        self.k, self.v, self.k_scale, self.v_scale, self.k_mean = k, v, k_scale, v_scale, k_mean
        # without keys, the means' sizes (no page size)
        n, h, ps, d = self._shape or (k_mean.shape[0], k_mean.shape[1], 0, k_mean.shape[2])
        self._view = _CacheView(
            ta_cache(*(t.data_ptr() if t is not None else None
                       for t in (k, v, k_scale, v_scale, k_mean))),
            self._strides, (n, h, ps, d), -1 if self._fmt is None else self._fmt, self._dev,
            int(k_mean is not None))

    def __setattr__(self, name, value):
        if getattr(self, name, value) is not value:      # (cache.k *= 2 sets k itself)
            raise AttributeError(f"PagedCache.{name} cannot be exchanged: make a new PagedCache")
        object.__setattr__(self, name, value)


def make_cache(p: ta_cache_params, device="cuda", layout: str = "hnd",
               means: bool = True) -> PagedCache:
    """A new cache for ``p``: zeroed pages, head-major ("hnd": [n_pages, Hkv,
    page_size, d]) or token-major ("nhd": [n_pages, page_size, Hkv, d])."""
    if layout not in ("hnd", "nhd"):
        raise ValueError(f"layout: expected 'hnd' or 'nhd', got {layout!r}")
    fp8 = p.format == TA_CACHE_FP8
    dt = torch.float8_e4m3fn if fp8 else torch.bfloat16
    a, b = (p.Hkv, p.page_size) if layout == "hnd" else (p.page_size, p.Hkv)

    def codes():
        x = torch.zeros((p.n_pages, a, b, p.d), dtype=torch.uint8 if fp8 else dt, device=device)
        x = x.view(dt) if fp8 else x
        return x if layout == "hnd" else x.transpose(1, 2)

    def scales():
        return torch.ones((p.n_pages, p.Hkv, p.page_size), device=device) if fp8 else None

    return PagedCache(codes(), codes(), scales(), scales(),
                      torch.zeros((p.n_pages, p.Hkv, p.d), device=device) if means else None)


def cache_workspace_bytes(p: ta_cache_params) -> int:
    return int(_fn("tiered_attn_cache_workspace_bytes")(ctypes.byref(p)))


def alloc_cache_workspace(p: ta_cache_params, device="cuda") -> torch.Tensor:
    """A workspace for every cached-attention call with ``p``, ready for use
    on the current stream."""
    n = cache_workspace_bytes(p)
    if n == 0:
        raise TieredAttnError("tiered_attn_cache_workspace_bytes", _b.TA_ERR_INVALID_ARG)
    ws = torch.empty(n, dtype=torch.uint8, device=device)
    with torch.cuda.device(ws.device):
        init_cache_workspace(ws)
    return ws


def init_cache_workspace(ws: torch.Tensor, stream=None) -> None:
    """Clear a workspace: before its first use, and to forget its status."""
    _check("tiered_attn_cache_init", _fn("tiered_attn_cache_init")(
        _b._ws(ws), ws.numel(), _b._stream(stream)))


def _plain(name, t, dtype, shape, dev) -> int:
    """Pointer of a contiguous tensor of this type and shape on device `dev`."""
    try:
        if t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    _refuse_type(name, t, dtype, dev)
    raise ValueError(f"{name}: expected a contiguous tensor of shape {tuple(shape)}, got "
                     f"{tuple(t.shape)} with strides {t.stride()}")


def _rows(name, t, shape, dev):
    """(pointer, row stride, head stride) of a bf16 [rows, heads, d] tensor, d
    contiguous."""
    try:
        if t.dtype is torch.bfloat16 and t.shape == shape and t.get_device() == dev:
            st, sh, sd = t.stride()
            if sd == 1:
                return t.data_ptr(), st, sh
    except AttributeError:
        pass
    _refuse_type(name, t, torch.bfloat16, dev)
    raise ValueError(f"{name}: expected shape {tuple(shape)} with the last dimension "
                     f"contiguous, got {tuple(t.shape)} with strides {t.stride()}")


def _refuse_type(name, t, dtype, dev) -> None:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor, got {type(t).__name__}")
    if t.get_device() != dev:
        raise ValueError(f"{name}: expected a tensor on device {dev}, got one on {t.device}")
    if t.dtype is not dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")


def _begin(p, cache, table, lens, ws, cu, kv: bool):
    """Checks shared by every call; (a copy of p with the cache's strides,
    device, pointers of table, lens and cu, pointer and size of ws)."""
    dev = cache._dev
    if dev < 0:
        raise ValueError("cache: expected CUDA tensors")
    if dev != torch._C._cuda_getDevice():
        raise ValueError(f"cache: on cuda:{dev}, but the library launches on the current device "
                         f"cuda:{torch._C._cuda_getDevice()}")
    S, W = p.S, p.max_pages
    q = ta_cache_params.from_buffer_copy(p)
    if kv:
        if cache._shape is None:
            raise ValueError("cache: has no keys and values")
        if cache._shape != (p.n_pages, p.Hkv, p.page_size, p.d) or cache._fmt != p.format:
            raise ValueError(f"cache: shape {cache._shape}, format {cache._fmt}, but the "
                             f"parameters say {(p.n_pages, p.Hkv, p.page_size, p.d)}, {p.format}")
        q.stride_page, q.stride_head, q.stride_slot = cache._strides
    try:
        rows, cols = table.shape
        q.stride_table, one = table.stride()
        ok = (table.dtype is torch.int32 and table.get_device() == dev and rows == S and
              cols >= W and one == 1)
    except (AttributeError, ValueError):
        ok = False
    if not ok:
        _refuse_type("table", table, torch.int32, dev)
        raise ValueError(f"table: expected [{S}, >= {W}] with contiguous rows, got "
                         f"{tuple(table.shape)} with strides {table.stride()}")
    ln = _plain("lens", lens, torch.int32, (S,), dev)
    c = None if cu is None else _plain("cu", cu, torch.int32, (S + 1,), dev)
    try:
        n = ws.numel()
    except AttributeError:
        n = 0
    return q, dev, table.data_ptr(), ln, c, _plain("ws", ws, torch.uint8, (n,), dev), n


def _stream_of(stream, dev) -> int:
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(dev)
    return _b._stream(stream)


def cache_append(p: ta_cache_params, cache: PagedCache, K, V, table, lens, ws, cu=None, cos=None,
                 sin=None, pos=None, Q=None, Q_out=None, stream=None) -> None:
    """Append the new tokens K, V bf16 [T, Hkv, d] to the cache, keys rotated
    by the table rows ``pos`` (their positions, where None) of ``cos`` and
    ``sin`` (f32 [rows, rot_dim / 2]); rotate Q [T, H, d] into ``Q_out`` (may
    be Q itself) with the same angles.  ``lens`` counts the new tokens."""
    st = _native().append(p, cache._view, K, V, table, lens, ws, cu, cos, sin, pos, Q,
                          Q_out, None if stream is None else _b._stream(stream))
    if st is not None:
        return _check("tiered_attn_cache_append", st)
    q, dev, tb, ln, c, w, n = _begin(p, cache, table, lens, ws, cu, True)
    T, d, rot = p.T, p.d, p.rot_dim
    shape = (T, p.Hkv, d)
    k, q.stride_k_t, q.stride_k_h = _rows("K", K, shape, dev)
    v, q.stride_v_t, q.stride_v_h = _rows("V", V, shape, dev)
    qi = qo = cp = sp = pp = None
    if Q is not None:
        shape = (T, p.H, d)
        qi, qt, qh = _rows("Q", Q, shape, dev)
        qo, ot, oh = _rows("Q_out", Q_out, shape, dev)
        if qi == qo and (qt, qh) != (ot, oh):
            raise ValueError("Q_out: shares Q's memory with other strides")
        q.stride_q_t, q.stride_q_h, q.stride_o_t, q.stride_o_h = qt, qh, ot, oh
    if rot:
        if not isinstance(cos, torch.Tensor):
            raise TypeError(f"cos: expected a torch.Tensor, got {type(cos).__name__}")
        shape = (len(cos), rot // 2)
        cp = _plain("cos", cos, torch.float32, shape, dev)
        sp = _plain("sin", sin, torch.float32, shape, dev)
        q.rot_rows = shape[0]
    if pos is not None:
        pp = _plain("pos", pos, torch.int32, (T,), dev)
    _check("tiered_attn_cache_append", _fn("tiered_attn_cache_append")(
        q, cache._view.c, k, v, qi, qo, cp, sp, pp, c, ln, tb, w, n, _stream_of(stream, dev)))


def cache_decode(p: ta_cache_params, cache: PagedCache, Q, table, lens, ws, O,
                 lse: Optional[torch.Tensor] = None, stream=None) -> None:
    """Attention of one new token for each sequence, Q bf16 [S, H, d], over
    its whole cache into O (and ``lse`` f32 [S, H])."""
    st = _native().decode(p, cache._view, Q, table, lens, ws, O, lse,
                          None if stream is None else _b._stream(stream))
    if st is not None:
        return _check("tiered_attn_cache_decode", st)
    q, dev, tb, ln, _, w, n = _begin(p, cache, table, lens, ws, None, True)
    shape = (p.T, p.H, p.d)
    qp, q.stride_q_t, q.stride_q_h = _rows("Q", Q, shape, dev)
    op, q.stride_o_t, q.stride_o_h = _rows("O", O, shape, dev)
    lp = None if lse is None else _plain("lse", lse, torch.float32, shape[:2], dev)
    _check("tiered_attn_cache_decode", _fn("tiered_attn_cache_decode")(
        q, cache._view.c, qp, ln, tb, op, lp, w, n, _stream_of(stream, dev)))


def cache_select(p: ta_cache_params, cache: PagedCache, Q, table, lens, ws, sel, cu=None,
                 stream=None) -> None:
    """The pages that each row reads: ``sel`` int32 [T, Hkv, n_select], page
    indices of the row's sequence in ascending order, then -1."""
    st = _native().select(p, cache._view, Q, table, lens, ws, sel, cu,
                          None if stream is None else _b._stream(stream))
    if st is not None:
        return _check("tiered_attn_cache_select", st)
    q, dev, tb, ln, c, w, n = _begin(p, cache, table, lens, ws, cu, False)
    if cache.k_mean is None or cache.k_mean.shape != (p.n_pages, p.Hkv, p.d):
        raise ValueError(f"cache: expected k_mean of shape {(p.n_pages, p.Hkv, p.d)}")
    qp, q.stride_q_t, q.stride_q_h = _rows("Q", Q, (p.T, p.H, p.d), dev)
    sl = _plain("sel", sel, torch.int32, (p.T, p.Hkv, p.n_select), dev)
    _check("tiered_attn_cache_select", _fn("tiered_attn_cache_select")(
        q, cache._view.c, qp, c, ln, tb, sl, w, n, _stream_of(stream, dev)))


def cache_sparse(p: ta_cache_params, cache: PagedCache, Q, sel, table, lens, ws, O, cu=None,
                 lse: Optional[torch.Tensor] = None, stream=None) -> None:
    """Attention of each row, Q bf16 [T, H, d], over the pages of its list
    ``sel`` into O (and ``lse`` f32 [T, H]).  O may not overlap Q."""
    st = _native().sparse(p, cache._view, Q, sel, table, lens, ws, O, cu, lse,
                          None if stream is None else _b._stream(stream))
    if st is not None:
        return _check("tiered_attn_cache_sparse", st)
    q, dev, tb, ln, c, w, n = _begin(p, cache, table, lens, ws, cu, True)
    shape = (p.T, p.H, p.d)
    qp, q.stride_q_t, q.stride_q_h = _rows("Q", Q, shape, dev)
    op, q.stride_o_t, q.stride_o_h = _rows("O", O, shape, dev)
    sl = _plain("sel", sel, torch.int32, (p.T, p.Hkv, p.n_select), dev)
    lp = None if lse is None else _plain("lse", lse, torch.float32, shape[:2], dev)
    _check("tiered_attn_cache_sparse", _fn("tiered_attn_cache_sparse")(
        q, cache._view.c, qp, sl, c, ln, tb, op, lp, w, n, _stream_of(stream, dev)))
