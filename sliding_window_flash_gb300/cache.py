"""Serving side of the binding: the paged 8-bit key/value cache, attention over it, its eviction by
accumulated attention weight, and the weights that a prompt's keys received (include/swa_cache.h).

    cache = SwaCache.empty(pages, Hkv, D, page=64)         # a pool of pages in device memory
    o, lse = swa_attn_fwd(q, k, v, window)                 # the prompt, as in training
    w = swa_attn_key_weights(q, k, lse, window)            # optional: what its keys received
    swa_cache_append(cache, table, lens, k, v, weight=w)   # lens: tokens cached before
    lens += N
    ...                                                    # then, for each new token:
    swa_cache_append(cache, table, lens, k1, v1)           # k1, v1 [B, Hkv, 1, D]
    o, lse = swa_cache_attn(q1, cache, table, lens, window, accumulate=True)
    lens += 1
    kept, lens = swa_cache_evict(cache, table, lens, spare, budget, recent)   # table = spare

``table`` [B, max_pages] and ``lens`` [B] are int32 CUDA tensors that the kernels read on the
device: nothing synchronises, and a captured step replays with their later contents.  Every call
runs on the current stream of the cache's device; a page number or length out of range is skipped
and reported by swa_check_device.
"""
from __future__ import annotations

import ctypes
import math
from typing import Optional

__all__ = [
    "SwaCache",
    "swa_cache_append",
    "swa_cache_attn",
    "swa_cache_attn_workspace_bytes",
    "swa_cache_evict",
    "swa_attn_key_weights",
    "swa_attn_key_weights_workspace_bytes",
]


class _CCache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("weight", ctypes.c_void_p),
                ("pages", ctypes.c_int), ("Hkv", ctypes.c_int), ("page", ctypes.c_int),
                ("D", ctypes.c_int)]


_c_int, _c_float, _vp = ctypes.c_int, ctypes.c_float, ctypes.c_void_p
_cp = ctypes.POINTER(_CCache)
SIGNATURES = {
    "swa_cache_append": (_c_int, [_cp, _vp, _c_int] + [_vp] * 5 + [_c_int] * 3 + [_vp]),
    "swa_cache_attn_workspace_bytes": (ctypes.c_size_t, [_c_int] * 8),
    "swa_cache_attn": (
        _c_int,
        [_cp, _vp, _c_int] + [_vp] * 5 + [_c_int] * 4 + [_c_float] + [_c_int] * 2 +
        [_vp, ctypes.c_size_t, _vp],
    ),
    "swa_cache_evict": (
        _c_int, [_cp, _vp, _c_int, _vp, _vp] + [_c_int] * 3 + [_vp, _vp, _c_int, _vp]),
    "swa_attn_key_weights_workspace_bytes": (ctypes.c_size_t, [_c_int] * 8),
    "swa_attn_key_weights": (
        _c_int, [_vp] * 4 + [_c_int] * 8 + [_c_float, _c_int, _vp, ctypes.c_size_t, _vp]),
}


_entries = {}


def _entry(name):
    """The library's entry point, loaded on first use."""
    fn = _entries.get(name)
    if fn is None:
        from . import load

        fn = _entries[name] = getattr(load(), name)
    return fn


def _check(t, name, shape, dtype, device):
    """Raises unless t is a contiguous CUDA tensor of this shape and dtype, on `device` if given."""
    import torch

    try:  # a good tensor costs four attribute reads
        if t.dtype is dtype and t.shape == shape and t.is_contiguous() and \
                (t.is_cuda if device is None else t.get_device() == device.index):
            return
    except AttributeError:
        pass
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    raise ValueError(f"{name} must be contiguous")


class SwaCache:
    """A pool of cache pages: k, v float8_e4m3fn [pages, Hkv, page, D], their scales k_scale, v_scale
    fp32 [pages, Hkv], and weight fp32 [pages, Hkv, page] (None for a cache never evicted from).
    The tensors are the caller's; this object only holds and checks them.  page is 32, 64 or 128,
    D 64, 128 or 256."""

    __slots__ = ("k", "v", "k_scale", "v_scale", "weight", "device")

    def __init__(self, k, v, k_scale, v_scale, weight=None):
        import torch

        if not isinstance(k, torch.Tensor) or k.dim() != 4:
            raise ValueError("k must be a 4-D tensor [pages, Hkv, page, D]")
        dev = k.device
        _check(k, "k", k.shape, torch.float8_e4m3fn, None)
        _check(v, "v", k.shape, torch.float8_e4m3fn, dev)
        _check(k_scale, "k_scale", k.shape[:2], torch.float32, dev)
        _check(v_scale, "v_scale", k.shape[:2], torch.float32, dev)
        if weight is not None:
            _check(weight, "weight", k.shape[:3], torch.float32, dev)
        put = object.__setattr__
        put(self, "k", k)
        put(self, "v", v)
        put(self, "k_scale", k_scale)
        put(self, "v_scale", v_scale)
        put(self, "weight", weight)
        put(self, "device", dev)

    def __setattr__(self, name, value):
        raise AttributeError("a SwaCache's tensors are fixed; make another for other tensors")

    @classmethod
    def empty(cls, pages: int, Hkv: int, D: int, page: int = 64, device=None, weight: bool = True):
        """A new pool of `pages` pages in device memory, zeroed."""
        import torch

        dev = torch.device("cuda", torch.cuda.current_device()) if device is None else device

        def codes():
            return torch.zeros((pages, Hkv, page, D), dtype=torch.uint8,
                               device=dev).view(torch.float8_e4m3fn)

        def scales():
            return torch.ones((pages, Hkv), dtype=torch.float32, device=dev)

        w = torch.zeros((pages, Hkv, page), dtype=torch.float32, device=dev) if weight else None
        return cls(codes(), codes(), scales(), scales(), w)

    @property
    def page(self) -> int:
        return self.k.shape[2]

    def _c(self):
        P, H, S, D = self.k.shape
        w = self.weight
        return _CCache(self.k.data_ptr(), self.v.data_ptr(), self.k_scale.data_ptr(),
                       self.v_scale.data_ptr(), None if w is None else w.data_ptr(), P, H, S, D)


def _tables(cache, table, lens, new):
    """(B, max_pages) after checking the int32 tables of a call."""
    import torch

    if not isinstance(cache, SwaCache):
        raise TypeError("cache must be a SwaCache")
    if not isinstance(table, torch.Tensor) or table.dim() != 2:
        raise ValueError("table must be a 2-D tensor [B, max_pages]")
    B, width = table.shape
    _check(table, "table", table.shape, torch.int32, cache.device)
    _check(lens, "lens", (B,), torch.int32, cache.device)
    if new is not None:
        _check(new, "new", (B,), torch.int32, cache.device)
    return B, width


def _window(window):
    """A window as the C int it becomes: one past every slot means the same however large."""
    return min(int(window), 2**31 - 1)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _space(workspace):
    """(address, bytes) of a workspace tensor."""
    if workspace is None:
        return None, 0
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _run(name, device, *args):
    """Calls entry point `name` on the device's current stream, with that device current."""
    import torch

    stream = torch._C._cuda_getCurrentRawStream(device.index)
    if device.index == torch.cuda.current_device():
        rc = _entry(name)(*args, stream)
    else:
        with torch.cuda.device(device):
            rc = _entry(name)(*args, stream)
    if rc != 0:
        from . import SwaError

        raise SwaError(rc, name)


def _dtype(t, name, fp32=False):
    import torch

    code = {torch.bfloat16: 0, torch.float16: 1}.get(t.dtype)
    if code is None and fp32 and t.dtype == torch.float32:
        code = 2
    if code is None:
        raise TypeError(f"{name} must be bfloat16{', float16 or float32' if fp32 else ' or float16'},"
                        f" got {t.dtype}")
    return code


def swa_cache_append(cache: SwaCache, table, lens, k, v, new=None, weight=None) -> None:
    """Quantises the new tokens' keys and values into the cache.

    k, v [B, Hkv, T, D] (bf16, fp16 or fp32): sequence b's first new[b] tokens (new int32 [B], or
    None: all T) go to slots lens[b], lens[b] + 1, ...  weight [B, Hkv, T] fp32: the accumulated
    attention weights they start with (None: zero).  The pages written must belong to one sequence.
    """
    import torch

    B, width = _tables(cache, table, lens, new)
    if not isinstance(k, torch.Tensor) or k.dim() != 4:
        raise ValueError("k must be a 4-D tensor [B, Hkv, T, D]")
    dt = _dtype(k, "k", fp32=True)
    T = k.shape[2]
    shape = (B, cache.k.shape[1], T, cache.k.shape[3])
    _check(k, "k", shape, k.dtype, cache.device)
    _check(v, "v", shape, k.dtype, cache.device)
    if weight is not None:
        _check(weight, "weight", shape[:3], torch.float32, cache.device)
    _run("swa_cache_append", cache.device, cache._c(), table.data_ptr(), width, lens.data_ptr(),
         _ptr(new), k.data_ptr(), v.data_ptr(), _ptr(weight), B, T, dt)


def swa_cache_attn_workspace_bytes(B: int, Hq: int, Hkv: int, T: int, D: int, max_pages: int,
                                   page: int, accumulate: bool = False) -> int:
    return int(_entry("swa_cache_attn_workspace_bytes")(B, Hq, Hkv, T, D, max_pages, page,
                                                        int(bool(accumulate))))


def swa_cache_attn(q, cache: SwaCache, table, lens, window: int, scale: Optional[float] = None,
                   new=None, accumulate: bool = False, out=None, lse=None, workspace=None):
    """Attention of the newest tokens over their cache: returns (o [B,Hq,T,D] in q's dtype, lse
    [B,Hq,T] fp32).

    q [B,Hq,T,D] bf16 or fp16, T <= 64: query t of sequence b sits at slot lens[b] + t (append its
    key and value first) and sees the window's slots up to its own.  new (int32 [B], or None) says
    how many of the T tokens are real; the rows of the others get o = 0, lse = -inf.  accumulate
    adds to cache.weight what each cached token received.  The workspace (of
    swa_cache_attn_workspace_bytes) is allocated here unless given.
    """
    import torch

    B, width = _tables(cache, table, lens, new)
    if not isinstance(q, torch.Tensor) or q.dim() != 4:
        raise ValueError("q must be a 4-D tensor [B, Hq, T, D]")
    dt = _dtype(q, "q")
    _, Hkv, page, D = cache.k.shape
    Hq, T = q.shape[1], q.shape[2]
    _check(q, "q", (B, Hq, T, D), q.dtype, cache.device)
    if out is None:
        out = torch.empty_like(q)
    else:
        _check(out, "out", (B, Hq, T, D), q.dtype, cache.device)
    if lse is None:
        lse = torch.empty((B, Hq, T), dtype=torch.float32, device=cache.device)
    else:
        _check(lse, "lse", (B, Hq, T), torch.float32, cache.device)
    if workspace is None:
        need = _entry("swa_cache_attn_workspace_bytes")(B, Hq, Hkv, T, D, width, page,
                                                        int(bool(accumulate)))
        workspace = torch.empty(need, dtype=torch.uint8, device=cache.device)
    _run("swa_cache_attn", cache.device, cache._c(), table.data_ptr(), width, lens.data_ptr(),
         _ptr(new), q.data_ptr(), out.data_ptr(), lse.data_ptr(), B, Hq, T, _window(window),
         1.0 / math.sqrt(D) if scale is None else float(scale), int(bool(accumulate)), dt,
         *_space(workspace))
    return out, lse


def swa_cache_evict(cache: SwaCache, table, lens, dst_table, budget: int, recent: int, kept=None,
                    lens_out=None):
    """Cuts every sequence and kv head to min(lens, budget) tokens: the `recent` last ones stay, and
    of the others those with the largest accumulated weight (equal: the earlier).  The survivors are
    written in order to the pages of dst_table [B, dst_pages], which must be none of table's; returns
    (kept [B,Hkv,budget] int32: their old slots, -1 behind the last; lens_out [B] int32)."""
    import torch

    B, width = _tables(cache, table, lens, None)
    if not isinstance(dst_table, torch.Tensor) or dst_table.dim() != 2:
        raise ValueError("dst_table must be a 2-D tensor [B, dst_pages]")
    _check(dst_table, "dst_table", (B, dst_table.shape[1]), torch.int32, cache.device)
    Hkv = cache.k.shape[1]
    shape = (B, Hkv, int(budget))
    if int(budget) < 1:
        raise ValueError("budget must be at least 1")
    if kept is None:
        kept = torch.empty(shape, dtype=torch.int32, device=cache.device)
    else:
        _check(kept, "kept", shape, torch.int32, cache.device)
    if lens_out is None:
        lens_out = torch.empty((B,), dtype=torch.int32, device=cache.device)
    else:
        _check(lens_out, "lens_out", (B,), torch.int32, cache.device)
    _run("swa_cache_evict", cache.device, cache._c(), table.data_ptr(), width, lens.data_ptr(),
         dst_table.data_ptr(), dst_table.shape[1], int(budget), int(recent), kept.data_ptr(),
         lens_out.data_ptr(), B)
    return kept, lens_out


def swa_attn_key_weights_workspace_bytes(B: int, Hq: int, Hkv: int, Lq: int, Lk: int, D: int,
                                         window: int, causal: bool = True) -> int:
    return int(_entry("swa_attn_key_weights_workspace_bytes")(B, Hq, Hkv, Lq, Lk, D,
                                                              _window(window), int(bool(causal))))


def swa_attn_key_weights(q, k, lse, window: int, scale: Optional[float] = None, causal: bool = True,
                         out=None, workspace=None):
    """The attention weight every key of a prompt received: fp32 [B,Hkv,Lk], the sum over the query
    heads of its kv head and the queries that see it of exp(scale <q, k> - lse).  q [B,Hq,Lq,D] and
    k [B,Hkv,Lk,D] in bf16 or fp16, lse [B,Hq,Lq] as swa_attn_fwd returned it for the same window,
    scale and causal.  The workspace (of swa_attn_key_weights_workspace_bytes) is allocated here
    unless given."""
    import torch

    for t in (q, k):
        if not isinstance(t, torch.Tensor) or t.dim() != 4:
            raise ValueError("q and k must be 4-D [B, H, L, D]")
    dt = _dtype(q, "q")
    B, Hq, Lq, D = q.shape
    Hkv, Lk = k.shape[1], k.shape[2]
    dev = q.device
    _check(q, "q", q.shape, q.dtype, None)
    _check(k, "k", (B, Hkv, Lk, D), q.dtype, dev)
    _check(lse, "lse", (B, Hq, Lq), torch.float32, dev)
    if out is None:
        out = torch.empty((B, Hkv, Lk), dtype=torch.float32, device=dev)
    else:
        _check(out, "out", (B, Hkv, Lk), torch.float32, dev)
    window, causal = _window(window), int(bool(causal))
    if workspace is None:
        need = _entry("swa_attn_key_weights_workspace_bytes")(B, Hq, Hkv, Lq, Lk, D, window, causal)
        if need:
            workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    _run("swa_attn_key_weights", dev, q.data_ptr(), k.data_ptr(), lse.data_ptr(), out.data_ptr(), B,
         Hq, Hkv, Lq, Lk, D, window, causal, 1.0 / math.sqrt(D) if scale is None else float(scale),
         dt, *_space(workspace))
    return out
