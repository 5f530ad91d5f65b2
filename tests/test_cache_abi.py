"""Host-only checks of the cache calls: every symbol of include/swa_cache.h is exported and bound,
and bad arguments are refused before anything is launched (no GPU needed)."""
import ctypes
import os
import re

import pytest
import torch

import sliding_window_flash_gb300 as swa
from sliding_window_flash_gb300 import cache as swa_cache_mod

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x10000  # 16-byte-aligned fake device address; never dereferenced by these calls


@pytest.fixture(scope="module")
def lib():
    from sliding_window_flash_gb300 import build as swa_build

    if not os.path.exists(swa.library_path()):
        swa_build.build()
    return swa.load()


def test_every_declared_symbol_is_exported(lib):
    text = open(os.path.join(ROOT, "include", "swa_cache.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = set(re.findall(r"\b(swa_[a-z_]+)\s*\(", text))
    assert names == set(swa_cache_mod.SIGNATURES)
    for name in names:
        assert hasattr(lib, name) and name in swa.SIGNATURES


def _c(k=FAKE, v=FAKE, ks=FAKE, vs=FAKE, w=FAKE, pages=9, H=2, page=64, D=128):
    return swa_cache_mod._CCache(k, v, ks, vs, w, pages, H, page, D)


CACHE_FAULTS = [
    (dict(k=0), 1), (dict(v=0), 1), (dict(ks=0), 1), (dict(vs=0), 1), (dict(pages=0), 1),
    (dict(H=0), 1), (dict(page=16), 2), (dict(page=48), 2), (dict(page=256), 2), (dict(D=96), 2),
    (dict(D=512), 2), (dict(k=FAKE + 8), 3), (dict(v=FAKE + 4), 3), (dict(ks=FAKE + 2), 3),
    (dict(vs=FAKE + 1), 3), (dict(w=FAKE + 4), 3), (dict(pages=1 << 30, H=2), 1),
]


def _append(lib, c=None, table=FAKE, width=4, lens=FAKE, new=0, k=FAKE, v=FAKE, w=0, B=2, T=3,
            dtype=0):
    return lib.swa_cache_append(c or _c(), table, width, lens, new, k, v, w, B, T, dtype, None)


def _attn(lib, c=None, table=FAKE, width=4, lens=FAKE, new=0, q=FAKE, o=FAKE, lse=FAKE, B=2, Hq=4,
          T=1, W=64, scale=0.1, acc=0, dtype=0, ws=FAKE, ws_bytes=1 << 40):
    return lib.swa_cache_attn(c or _c(), table, width, lens, new, q, o, lse, B, Hq, T, W, scale,
                              acc, dtype, ws, ws_bytes, None)


def _evict(lib, c=None, table=FAKE, width=4, lens=FAKE, dst=FAKE, room=2, budget=100, recent=10,
           kept=FAKE, out=FAKE, B=2):
    return lib.swa_cache_evict(c or _c(), table, width, lens, dst, room, budget, recent, kept, out,
                               B, None)


@pytest.mark.parametrize("kw,code", CACHE_FAULTS)
@pytest.mark.parametrize("call", [_append, _attn, _evict], ids=["append", "attn", "evict"])
def test_bad_caches(lib, call, kw, code):
    assert call(lib, c=_c(**kw)) == code


@pytest.mark.parametrize("call", [_append, _attn, _evict], ids=["append", "attn", "evict"])
def test_bad_tables(lib, call):
    assert call(lib, table=0) == 1 and call(lib, lens=0) == 1
    assert call(lib, width=0) == 1 and call(lib, B=0) == 1 and call(lib, B=70000) == 1
    assert call(lib, width=1 << 26) == 1  # slots past 31 bits
    assert call(lib, table=FAKE + 2) == 3 and call(lib, lens=FAKE + 1) == 3


@pytest.mark.parametrize("kw,code", [
    (dict(k=0), 1), (dict(v=0), 1), (dict(T=0), 1), (dict(dtype=3), 1), (dict(dtype=-1), 1),
    (dict(k=FAKE + 8), 3), (dict(v=FAKE + 8), 3), (dict(w=FAKE + 2), 3), (dict(new=FAKE + 2), 3),
    (dict(B=1 << 15, T=1 << 16), 1),
])
def test_append_refusals(lib, kw, code):
    assert _append(lib, **kw) == code


def test_weights_need_a_cache_that_holds_them(lib):
    assert _append(lib, c=_c(w=0), w=FAKE) == 1
    assert _attn(lib, c=_c(w=0), acc=1) == 1
    assert _evict(lib, c=_c(w=0)) == 1


@pytest.mark.parametrize("kw,code", [
    (dict(q=0), 1), (dict(o=0), 1), (dict(lse=0), 1), (dict(Hq=0), 1), (dict(Hq=3), 1),
    (dict(W=0), 1), (dict(T=0), 1), (dict(T=65), 1), (dict(scale=0.0), 1),
    (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1), (dict(acc=2), 1),
    (dict(dtype=2), 1), (dict(q=FAKE + 8), 3), (dict(o=FAKE + 8), 3), (dict(lse=FAKE + 2), 3),
    (dict(new=FAKE + 2), 3),
])
def test_attn_refusals(lib, kw, code):
    assert _attn(lib, **kw) == code


def test_attn_workspace(lib):
    size = lib.swa_cache_attn_workspace_bytes
    for bad in ((0, 4, 2, 1, 128, 4, 64, 0), (2, 3, 2, 1, 128, 4, 64, 0), (2, 4, 2, 0, 128, 4, 64, 0),
                (2, 4, 2, 65, 128, 4, 64, 0), (2, 4, 2, 1, 96, 4, 64, 0), (2, 4, 2, 1, 128, 0, 64, 0),
                (2, 4, 2, 1, 128, 4, 48, 0)):
        assert size(*bad) == 0
    for acc in (0, 1):
        need = size(2, 4, 2, 1, 128, 4, 64, acc)
        if need:
            assert _attn(lib, acc=acc, ws_bytes=need - 1) == 6
            assert _attn(lib, acc=acc, ws=0) == 6
            assert _attn(lib, acc=acc, ws=FAKE + 8) == 3


@pytest.mark.parametrize("kw,code", [
    (dict(dst=0), 1), (dict(kept=0), 1), (dict(out=0), 1), (dict(budget=0), 1),
    (dict(recent=-1), 1), (dict(recent=101), 1), (dict(room=0), 1), (dict(room=1), 1),
    (dict(dst=FAKE + 2), 3), (dict(kept=FAKE + 2), 3), (dict(out=FAKE + 2), 3),
])
def test_evict_refusals(lib, kw, code):
    assert _evict(lib, **kw) == code


def test_evict_refuses_its_own_table_as_destination(lib):
    assert _evict(lib, dst=FAKE, table=FAKE) == 1


@pytest.mark.parametrize("call", [_append, _attn, _evict], ids=["append", "attn", "evict"])
def test_slots_stay_below_thirty_bits(lib, call):
    assert call(lib, width=1 << 24) == 1
    assert lib.swa_cache_attn_workspace_bytes(2, 4, 2, 1, 128, 1 << 24, 64, 0) == 0
    assert lib.swa_cache_attn_workspace_bytes(2, 4, 2, 1, 128, (1 << 24) - 1, 64, 0) > 0


def _weights(lib, q=FAKE, k=FAKE, lse=FAKE, w=FAKE, B=1, Hq=4, H=2, Lq=16, Lk=20, D=64, W=4,
             causal=1, scale=0.1, dtype=0, ws=FAKE, ws_bytes=1 << 40):
    return lib.swa_attn_key_weights(q, k, lse, w, B, Hq, H, Lq, Lk, D, W, causal, scale, dtype, ws,
                                    ws_bytes, None)


@pytest.mark.parametrize("kw,code", [
    (dict(q=0), 1), (dict(k=0), 1), (dict(lse=0), 1), (dict(w=0), 1), (dict(B=0), 1),
    (dict(Hq=3), 1), (dict(Lq=0), 1), (dict(Lq=21), 1), (dict(W=0), 1), (dict(causal=2), 1),
    (dict(scale=-1.0), 1), (dict(dtype=2), 1), (dict(D=96), 2), (dict(q=FAKE + 8), 3),
    (dict(w=FAKE + 2), 3), (dict(lse=FAKE + 1), 3), (dict(k=FAKE + 8), 3),
    (dict(B=1 << 16, Lq=1 << 14, Lk=1 << 14), 1),
])
def test_key_weights_refusals(lib, kw, code):
    assert _weights(lib, **kw) == code


def test_key_weights_workspace(lib):
    size = lib.swa_attn_key_weights_workspace_bytes
    need = size(1, 4, 2, 600, 700, 64, 4, 1)
    pieces = need / (2 * 700 * 4)
    assert pieces >= 2 and need % 256 == 0
    big = dict(Lq=600, Lk=700)
    assert _weights(lib, ws_bytes=need - 1, **big) == 6
    assert _weights(lib, ws=0, **big) == 6 and _weights(lib, ws=FAKE + 8, **big) == 3
    for bad in ((0, 4, 2, 16, 20, 64, 4, 1), (1, 3, 2, 16, 20, 64, 4, 1), (1, 4, 2, 21, 20, 64, 4, 1),
                (1, 4, 2, 16, 20, 96, 4, 1), (1, 4, 2, 16, 20, 64, 0, 1), (1, 4, 2, 16, 20, 64, 4, 2)):
        assert size(*bad) == 0
    # one walk per block of keys needs none
    assert size(1, 32, 16, 1 << 20, 1 << 20, 128, 1024, 1) == 0


def test_binding_refuses_what_is_not_on_the_gpu():
    k = torch.zeros((2, 1, 64, 64), dtype=torch.uint8).view(torch.float8_e4m3fn)
    s = torch.ones((2, 1))
    with pytest.raises(ValueError):
        swa.SwaCache(k, k, s, s)
    with pytest.raises(ValueError):
        swa.SwaCache(torch.zeros(3), k, s, s)
    with pytest.raises(TypeError):
        swa.swa_cache_append("cache", None, None, None, None)
    q = torch.zeros((1, 2, 8, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        swa.swa_attn_key_weights(q, q, torch.zeros((1, 2, 8)), 4)
    with pytest.raises(TypeError):
        swa.swa_attn_key_weights(q.float(), q.float(), torch.zeros((1, 2, 8)), 4)


def test_struct_matches_the_header():
    """The fields of swa_cache in the header, in order, are the binding's."""
    text = open(os.path.join(ROOT, "include", "swa_cache.h")).read()
    body = re.sub(r"/\*.*?\*/", "", text.split("typedef struct swa_cache {")[1].split("}")[0],
                  flags=re.S)
    names = re.findall(r"(?:void\*|float\*|int) (\w+);", body)
    assert names == [n for n, _ in swa_cache_mod._CCache._fields_]
    assert ctypes.sizeof(swa_cache_mod._CCache) == 5 * 8 + 4 * 4


def test_calls_run_on_the_caches_gpu(monkeypatch):
    """A call makes the tensors' GPU current, takes that GPU's stream, and leaves the current one."""
    now, seen = [0], []

    class Device:
        def __init__(self, index):
            self.index = index

        def __enter__(self):
            self.was, now[0] = now[0], self.index

        def __exit__(self, *_):
            now[0] = self.was

    class Names:
        stream = staticmethod(lambda index: 1000 + index)
        current_device = staticmethod(lambda: now[0])

    monkeypatch.setattr(swa_cache_mod, "_t", Names)
    monkeypatch.setattr(torch.cuda, "device", Device)
    rc = [0]

    def entry(*args):
        seen.append((now[0], args))
        return rc[0]

    monkeypatch.setitem(swa_cache_mod._entries, "swa_cache_append", entry)
    swa_cache_mod._run("swa_cache_append", 0, 7)
    swa_cache_mod._run("swa_cache_append", 3, 8)
    assert seen == [(0, (7, 1000)), (3, (8, 1003))] and now[0] == 0
    rc[0] = 1
    with pytest.raises(swa.SwaError):
        swa_cache_mod._run("swa_cache_append", 3, 8)
    assert now[0] == 0
