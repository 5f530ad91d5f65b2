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

Where the model has sinks, the prompt's and the tokens' calls take the same ``sinks=``.  Where the tables
of a batch begin with the same pages (a system prompt's), ``shared=`` says how many, and their slots are
walked once for the batch; the rows behind are each sequence's own.

``table`` [B, max_pages] and ``lens`` [B] are int32 CUDA tensors that the kernels read on the
device: nothing synchronises, and a captured step replays with their later contents.  Every call
runs on the current stream of the cache's device; a page number or length out of range is skipped
and reported by swa_check_device.
"""
from __future__ import annotations

import ctypes
import functools
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
    "swa_cache_attn_window_workspace_bytes": (ctypes.c_size_t, [_c_int] * 9),
    "swa_cache_attn": (
        _c_int,
        [_cp, _vp, _c_int] + [_vp] * 5 + [_c_int] * 4 + [_c_float] + [_c_int] * 2 +
        [_vp, ctypes.c_size_t, _vp],
    ),
    "swa_cache_attn_sinks_workspace_bytes": (ctypes.c_size_t, [_c_int] * 10),
    "swa_cache_attn_sinks": (
        _c_int,
        [_cp, _vp, _c_int] + [_vp] * 5 + [_c_int] * 5 + [_c_float] + [_c_int] * 2 +
        [_vp, ctypes.c_size_t, _vp],
    ),
    "swa_cache_attn_shared_workspace_bytes": (ctypes.c_size_t, [_c_int] * 11),
    "swa_cache_attn_shared": (
        _c_int,
        [_cp, _vp, _c_int] + [_vp] * 5 + [_c_int] * 6 + [_c_float] + [_c_int] * 2 +
        [_vp, ctypes.c_size_t, _vp],
    ),
    "swa_cache_evict": (
        _c_int, [_cp, _vp, _c_int, _vp, _vp] + [_c_int] * 3 + [_vp, _vp, _c_int, _vp]),
    "swa_attn_key_weights_workspace_bytes": (ctypes.c_size_t, [_c_int] * 8),
    "swa_attn_key_weights": (
        _c_int, [_vp] * 4 + [_c_int] * 8 + [_c_float, _c_int, _vp, ctypes.c_size_t, _vp]),
    "swa_attn_key_weights_sinks_workspace_bytes": (ctypes.c_size_t, [_c_int] * 9),
    "swa_attn_key_weights_sinks": (
        _c_int, [_vp] * 4 + [_c_int] * 9 + [_c_float, _c_int, _vp, ctypes.c_size_t, _vp]),
}


class _Torch:
    """torch's names that every call needs, looked up once (the package imports torch lazily).
    Tensors are made by empty: between two launches it takes 2.7 us on a Grace core, new_empty 4.1."""

    def __getattr__(self, name):
        if name in _SHORT:  # these need the library, the others do not
            self.__dict__[name] = _short_way()[name]
            return self.__dict__[name]
        import torch

        self.__dict__.update(
            f8=torch.float8_e4m3fn, f32=torch.float32, i32=torch.int32, u8=torch.uint8,
            kinds={torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}, Tensor=torch.Tensor,
            empty=torch.empty, empty_like=torch.empty_like, stream=torch._C._cuda_getCurrentRawStream,
            current_device=torch._C._cuda_getDevice)
        return self.__dict__[name]


_SHORT = ("pool", "attn", "fwd", "bwd")


def _short_way():
    """The calls of _swa_torch.so: each answers a call whose arguments are plainly in order, with what it
    returns or the status of an error, and None for any other.  Without the module every call is another, and
    so with one that was compiled for another torch or Python: it would read their objects by old layouts."""
    import torch

    from . import library_path
    from .build import built_for

    try:
        from . import _swa_torch as m

        if getattr(m, "built_for", None) != built_for(torch.__version__):
            raise ImportError("_swa_torch.so was compiled for another torch or Python")
        lib = ctypes.CDLL(library_path())
        m.use(*[ctypes.cast(getattr(lib, name), _vp).value for name in (
            "swa_cache_attn", "swa_cache_attn_sinks", "swa_cache_attn_shared",
            "swa_cache_attn_shared_workspace_bytes", "swa_attn_fwd_sinks", "swa_attn_bwd_sinks",
            "swa_attn_sinks_workspace_bytes")])
        return {"pool": m.pool, "attn": m.cache_attn, "fwd": m.fwd, "bwd": m.bwd}
    except (ImportError, OSError):  # no module, or no library: what is missing is said by the Python way
        return dict.fromkeys(_SHORT, lambda *_: None)


def _raise(rc, name):
    from . import SwaError

    raise SwaError(rc, name)


_t = _Torch()
_entries = {}


def _entry(name):
    """The library's entry point, loaded on first use."""
    fn = _entries.get(name)
    if fn is None:
        from . import load

        fn = _entries[name] = getattr(load(), name)
    return fn


def _good(t, shape, dtype, index):
    """Whether t is a contiguous tensor of this shape and dtype on GPU `index`: the few reads that a
    good tensor costs on every call."""
    try:
        return (t.dtype is dtype and t.get_device() == index and t.shape == shape and
                t.is_contiguous())
    except AttributeError:
        return False


def _check(t, name, shape, dtype, device):
    """Raises unless t is a contiguous CUDA tensor of this shape and dtype, on `device` if given."""
    import torch

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
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


_put = object.__setattr__


class SwaCache:
    """A pool of cache pages: k, v float8_e4m3fn [pages, Hkv, page, D], their scales k_scale, v_scale
    fp32 [pages, Hkv], and weight fp32 [pages, Hkv, page] (None for a cache never evicted from).
    The tensors are the caller's; this object only holds and checks them.  page is 32, 64 or 128,
    D 64, 128 or 256."""

    __slots__ = ("held",)
    k, v, k_scale, v_scale, weight, device, shape = (
        property(lambda self, i=i: self.held[i]) for i in range(7))

    def __init__(self, k, v, k_scale, v_scale, weight=None):
        t = _t
        held = t.pool(k, v, k_scale, v_scale, weight)
        if held is not None:
            _put(self, "held", held)
            return
        if not isinstance(k, t.Tensor) or k.dim() != 4:
            raise ValueError("k must be a 4-D tensor [pages, Hkv, page, D]")
        dev, shape = k.device, tuple(k.shape)
        f8, f32, index, blocks = t.f8, t.f32, dev.index, shape[:2]
        if not (index is not None and _good(k, shape, f8, index) and _good(v, shape, f8, index) and
                _good(k_scale, blocks, f32, index) and _good(v_scale, blocks, f32, index) and
                (weight is None or _good(weight, shape[:3], f32, index))):
            _check(k, "k", shape, f8, None)
            _check(v, "v", shape, f8, dev)
            _check(k_scale, "k_scale", blocks, f32, dev)
            _check(v_scale, "v_scale", blocks, f32, dev)
            if weight is not None:
                _check(weight, "weight", shape[:3], f32, dev)
        _put(self, "held", (k, v, k_scale, v_scale, weight, dev, shape))

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
        return self.shape[2]

    def _c(self):
        k, v, ks, vs, w, _, shape = self.held
        return _CCache(k.data_ptr(), v.data_ptr(), ks.data_ptr(), vs.data_ptr(),
                       None if w is None else w.data_ptr(), *shape)


def _tables(cache, table, lens, new):
    """(B, max_pages, GPU index) after checking the int32 tables of a call."""
    if type(cache) is not SwaCache:
        raise TypeError("cache must be a SwaCache")
    t, dev = _t, cache.held[5]
    if not isinstance(table, t.Tensor) or table.dim() != 2:
        raise ValueError("table must be a 2-D tensor [B, max_pages]")
    shape, index, i32 = tuple(table.shape), dev.index, t.i32
    B = shape[:1]
    if not (_good(table, shape, i32, index) and _good(lens, B, i32, index) and
            (new is None or _good(new, B, i32, index))):
        _check(table, "table", shape, i32, dev)
        _check(lens, "lens", B, i32, dev)
        if new is not None:
            _check(new, "new", B, i32, dev)
    return shape[0], shape[1], index


def _int32(x):
    """The C int nearest to x: what an int does not hold must not wrap to another number.  A window past
    every slot means the same however large; what else is out of range is refused."""
    x = int(x)
    return x if -2**31 <= x < 2**31 else 2**31 - 1 if x > 0 else -2**31


def _ptr(t):
    return None if t is None else t.data_ptr()


def _space(workspace, device):
    """(address, bytes) of a caller's workspace: all of its bytes are there, on `device`."""
    if not isinstance(workspace, _t.Tensor):
        raise TypeError("workspace must be a torch.Tensor")
    if workspace.device != device:
        raise ValueError(f"workspace is on {workspace.device}, expected {device}")
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _on(index, name, *args):
    """Calls entry point `name` with GPU `index` current."""
    if index == _t.current_device():
        return _entry(name)(*args)
    import torch

    with torch.cuda.device(index):
        return _entry(name)(*args)


def _run(name, index, *args):
    """Calls entry point `name` on the current stream of GPU `index`, with that GPU current."""
    rc = _on(index, name, *args, _t.stream(index))
    if rc != 0:
        _raise(rc, name)


def _dtype(t, name, fp32=False):
    code = _t.kinds.get(t.dtype, 3)
    if code < 2 or fp32 and code == 2:
        return code
    raise TypeError(f"{name} must be bfloat16{', float16 or float32' if fp32 else ' or float16'}, "
                    f"got {t.dtype}")


def swa_cache_append(cache: SwaCache, table, lens, k, v, new=None, weight=None) -> None:
    """Quantises the new tokens' keys and values into the cache.

    k, v [B, Hkv, T, D] (bf16, fp16 or fp32): sequence b's first new[b] tokens (new int32 [B], or
    None: all T) go to slots lens[b], lens[b] + 1, ...  weight [B, Hkv, T] fp32: the accumulated
    attention weights they start with (None: zero).  The pages written must belong to one sequence.
    """
    B, width, index = _tables(cache, table, lens, new)
    if not isinstance(k, _t.Tensor) or k.dim() != 4:
        raise ValueError("k must be a 4-D tensor [B, Hkv, T, D]")
    dt, kind = _dtype(k, "k", fp32=True), k.dtype
    T = k.shape[2]
    shape = (B, cache.shape[1], T, cache.shape[3])
    if not (_good(k, shape, kind, index) and _good(v, shape, kind, index) and
            (weight is None or _good(weight, shape[:3], _t.f32, index))):
        _check(k, "k", shape, kind, cache.device)
        _check(v, "v", shape, kind, cache.device)
        if weight is not None:
            _check(weight, "weight", shape[:3], _t.f32, cache.device)
    _run("swa_cache_append", index, cache._c(), table.data_ptr(), width, lens.data_ptr(),
         _ptr(new), k.data_ptr(), v.data_ptr(), _ptr(weight), B, T, dt)


# A workspace's size follows the number of the GPU's SMs, so it is asked for, and kept, for that GPU.
@functools.lru_cache(maxsize=256)
def _attn_space(index, *sizes):
    return int(_on(index, "swa_cache_attn_shared_workspace_bytes", *sizes))


@functools.lru_cache(maxsize=256)
def _weights_space(index, *sizes):
    sinks = "_sinks" if len(sizes) == 9 else ""
    return int(_on(index, f"swa_attn_key_weights{sinks}_workspace_bytes", *sizes))


def swa_cache_attn_workspace_bytes(B: int, Hq: int, Hkv: int, T: int, D: int, max_pages: int,
                                   page: int, accumulate: bool = False,
                                   window: Optional[int] = None, sinks: int = 0,
                                   shared: int = 0) -> int:
    """Bytes of swa_cache_attn's workspace on the current GPU, for this window or (None) for any."""
    sizes, acc = (B, Hq, Hkv, T, D, max_pages, page), int(bool(accumulate))
    if shared:
        return int(_entry("swa_cache_attn_shared_workspace_bytes")(
            *sizes, 2**31 - 1 if window is None else _int32(window), _int32(sinks), _int32(shared), acc))
    if window is None:  # the whole table, sinks included
        return int(_entry("swa_cache_attn_workspace_bytes")(*sizes, acc))
    if not sinks:
        return int(_entry("swa_cache_attn_window_workspace_bytes")(*sizes, _int32(window), acc))
    return int(_entry("swa_cache_attn_sinks_workspace_bytes")(*sizes, _int32(window), _int32(sinks), acc))


def swa_cache_attn(q, cache: SwaCache, table, lens, window: int, scale: Optional[float] = None,
                   new=None, accumulate: bool = False, out=None, lse=None, workspace=None,
                   sinks: int = 0, shared: int = 0):
    """Attention of the newest tokens over their cache: returns (o [B,Hq,T,D] in q's dtype, lse
    [B,Hq,T] fp32).

    q [B,Hq,T,D] bf16 or fp16, T <= 64: query t of sequence b sits at slot lens[b] + t (append its
    key and value first) and sees the window's slots up to its own, and behind the window the first
    `sinks` slots.  new (int32 [B], or None) says
    how many of the T tokens are real; the rows of the others get o = 0, lse = -inf.  accumulate
    adds to cache.weight what each cached token received.  shared says that the first `shared` entries
    of all tables are the same pages: their slots are walked once for all sequences (without
    accumulate).  The workspace (of swa_cache_attn_workspace_bytes, for this window, sinks and shared;
    without shared also for any window) is allocated here unless given.
    """
    if type(cache) is SwaCache:
        done = _t.attn(cache.held, q, table, lens, new, out, lse, workspace, window, scale, accumulate, sinks,
                       shared)
        if type(done) is tuple:
            return done
        if done is not None:
            _raise(done, "swa_cache_attn" + ("_shared" if shared else "_sinks" if sinks else ""))
    B, width, index = _tables(cache, table, lens, new)
    dev, (_, Hkv, page, D) = cache.held[5:]
    if not isinstance(q, _t.Tensor) or q.dim() != 4:
        raise ValueError("q must be a 4-D tensor [B, Hq, T, D]")
    dt, kind, f32 = _dtype(q, "q"), q.dtype, _t.f32
    _, Hq, T, _ = q.shape
    shape = (B, Hq, T, D)
    if not _good(q, shape, kind, index):
        _check(q, "q", shape, kind, dev)
    if out is None:
        out = _t.empty_like(q)
    elif not _good(out, shape, kind, index):
        _check(out, "out", shape, kind, dev)
    if lse is None:
        lse = _t.empty(shape[:3], dtype=f32, device=dev)
    elif not _good(lse, shape[:3], f32, index):
        _check(lse, "lse", shape[:3], f32, dev)
    window, accumulate = _int32(window), int(bool(accumulate))
    sinks, shared = sinks and _int32(sinks), shared and _int32(shared)
    if workspace is None:
        need = _attn_space(index, B, Hq, Hkv, T, D, width, page, window, sinks, shared, accumulate)
        workspace = _t.empty(need, dtype=_t.u8, device=dev)
        space = workspace.data_ptr(), need
    else:
        space = _space(workspace, dev)
    scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    args = (cache._c(), table.data_ptr(), width, lens.data_ptr(), _ptr(new), q.data_ptr(),
            out.data_ptr(), lse.data_ptr(), B, Hq, T, window)
    if shared:
        _run("swa_cache_attn_shared", index, *args, sinks, shared, scale, accumulate, dt, *space)
    elif sinks:
        _run("swa_cache_attn_sinks", index, *args, sinks, scale, accumulate, dt, *space)
    else:
        _run("swa_cache_attn", index, *args, scale, accumulate, dt, *space)
    return out, lse


def swa_cache_evict(cache: SwaCache, table, lens, dst_table, budget: int, recent: int, kept=None,
                    lens_out=None):
    """Cuts every sequence and kv head to min(lens, budget) tokens: the `recent` last ones stay, and
    of the others those with the largest accumulated weight (equal: the earlier).  The survivors are
    written in order to the pages of dst_table [B, dst_pages], which must be none of table's; returns
    (kept [B,Hkv,budget] int32: their old slots, -1 behind the last; lens_out [B] int32, which may be
    given as lens itself).  A sequence whose length is out of range keeps nothing: lens_out 0.  Sinks are
    tokens like others here, and sinks= counts what is cached: where a model has them, their weights are set
    to infinity before, and they stay first in every head."""
    B, width, index = _tables(cache, table, lens, None)
    if not isinstance(dst_table, _t.Tensor) or dst_table.dim() != 2:
        raise ValueError("dst_table must be a 2-D tensor [B, dst_pages]")
    budget, i32 = int(budget), _t.i32
    if not 1 <= budget < 2**30:  # slots of a table
        raise ValueError("budget must be at least 1 and below 2^30")
    room = (B, dst_table.shape[1])
    if not _good(dst_table, room, i32, index):
        _check(dst_table, "dst_table", room, i32, cache.device)
    shape = (B, cache.shape[1], budget)
    if kept is None:
        kept = _t.empty(shape, dtype=i32, device=cache.device)
    elif not _good(kept, shape, i32, index):
        _check(kept, "kept", shape, i32, cache.device)
    if lens_out is None:
        lens_out = _t.empty_like(lens)
    elif not _good(lens_out, (B,), i32, index):
        _check(lens_out, "lens_out", (B,), i32, cache.device)
    _run("swa_cache_evict", index, cache._c(), table.data_ptr(), width, lens.data_ptr(),
         dst_table.data_ptr(), room[1], budget, _int32(recent), kept.data_ptr(), lens_out.data_ptr(), B)
    return kept, lens_out


def swa_attn_key_weights_workspace_bytes(B: int, Hq: int, Hkv: int, Lq: int, Lk: int, D: int,
                                         window: int, causal: bool = True, sinks: int = 0) -> int:
    """Bytes of swa_attn_key_weights' workspace on the current GPU."""
    sizes = B, Hq, Hkv, Lq, Lk, D, _int32(window)
    if sinks:
        return int(_entry("swa_attn_key_weights_sinks_workspace_bytes")(*sizes, _int32(sinks),
                                                                        int(bool(causal))))
    return int(_entry("swa_attn_key_weights_workspace_bytes")(*sizes, int(bool(causal))))


def swa_attn_key_weights(q, k, lse, window: int, scale: Optional[float] = None, causal: bool = True,
                         out=None, workspace=None, sinks: int = 0):
    """The attention weight every key of a prompt received: fp32 [B,Hkv,Lk], the sum over the query
    heads of its kv head and the queries that see it of exp(scale <q, k> - lse).  q [B,Hq,Lq,D] and
    k [B,Hkv,Lk,D] in bf16 or fp16, lse [B,Hq,Lq] as swa_attn_fwd returned it for the same window,
    scale, causal and sinks.  The workspace (of swa_attn_key_weights_workspace_bytes) is allocated here
    unless given."""
    for t in (q, k):
        if not isinstance(t, _t.Tensor) or t.dim() != 4:
            raise ValueError("q and k must be 4-D [B, H, L, D]")
    dt, kind, f32 = _dtype(q, "q"), q.dtype, _t.f32
    B, Hq, Lq, D = q.shape
    Hkv, Lk = k.shape[1], k.shape[2]
    dev = q.device
    index = dev.index
    if not (index is not None and _good(q, q.shape, kind, index) and
            _good(k, (B, Hkv, Lk, D), kind, index) and _good(lse, (B, Hq, Lq), f32, index)):
        _check(q, "q", q.shape, kind, None)
        _check(k, "k", (B, Hkv, Lk, D), kind, dev)
        _check(lse, "lse", (B, Hq, Lq), f32, dev)
    if out is None:
        out = _t.empty((B, Hkv, Lk), dtype=f32, device=dev)
    elif not _good(out, (B, Hkv, Lk), f32, index):
        _check(out, "out", (B, Hkv, Lk), f32, dev)
    window, causal = _int32(window), int(bool(causal))
    name, reach = "swa_attn_key_weights", (window, causal)
    if sinks:
        name, reach = "swa_attn_key_weights_sinks", (window, _int32(sinks), causal)
    space = None, 0
    if workspace is not None:
        space = _space(workspace, dev)
    else:
        need = _weights_space(index, B, Hq, Hkv, Lq, Lk, D, *reach)
        if need:
            workspace = _t.empty(need, dtype=_t.u8, device=dev)
            space = workspace.data_ptr(), need
    _run(name, index, q.data_ptr(), k.data_ptr(), lse.data_ptr(), out.data_ptr(), B, Hq, Hkv, Lq, Lk, D,
         *reach, 1.0 / math.sqrt(D) if scale is None else float(scale), dt, *space)
    return out
