"""The paged-cache entry points' refusals and sizes, on the CPU: everything here is decided on the
host before any work is enqueued (the pointers are never dereferenced)."""
import ctypes

import pytest
import torch

from local_linear_attention_gb300 import build as lla_build

OK, INVALID, UNSUPPORTED = 0, 1, 2


@pytest.fixture(scope="module")
def lla():
    lla_build.build()
    from local_linear_attention_gb300 import binding
    return binding


class CacheStruct(ctypes.Structure):
    """lla_paged_cache, field by field."""
    _fields_ = [(n, ctypes.c_void_p) for n in ("k_pages", "v_pages", "mass", "page_table", "lens")] + \
        [(n, ctypes.c_int) for n in ("num_seqs", "kv_heads", "page_size", "max_pages", "num_pages", "d", "dv",
                                     "dtype")] + [("reserved", ctypes.c_int * 2)]


class QueryStruct(ctypes.Structure):
    """lla_paged_query, field by field."""
    _fields_ = [(n, ctypes.c_void_p) for n in ("q", "r", "out", "lse", "starts")] + \
        [(n, ctypes.c_int) for n in ("tokens", "max_new", "q_heads")] + [("h", ctypes.c_float)] + \
        [(n, ctypes.c_int) for n in ("window", "sinks", "track_mass", "path")] + [("reserved", ctypes.c_int * 2)]


def cache(lla, **kw):
    f = dict(k_pages=256, v_pages=512, mass=768, page_table=1024, lens=1280, num_seqs=2, kv_heads=2,
             page_size=16, max_pages=8, num_pages=20, d=64, dv=64, dtype=1)
    f.update(kw)
    return CacheStruct(**f)


def query(lla, **kw):
    f = dict(q=256, r=None, out=512, lse=None, starts=768, tokens=4, max_new=2, q_heads=4, h=8.0, window=0,
             sinks=0, track_mass=0, path=0)
    f.update(kw)
    return QueryStruct(**f)


def attend(lla, c, q, ws=None, n=0):
    return lla._load().lla_paged_attention(ctypes.byref(c), ctypes.byref(q), ws, n, None)


def test_struct_sizes(lla):
    """The binding packs the same bytes."""
    assert lla._CACHE.size == ctypes.sizeof(CacheStruct) and lla._QUERY.size == ctypes.sizeof(QueryStruct)
    got = CacheStruct.from_buffer_copy(lla._CACHE.pack(*range(15)))
    flat = [getattr(got, f[0]) or 0 for f in CacheStruct._fields_[:-1]] + list(got.reserved)
    assert flat == list(range(15))
    got = QueryStruct.from_buffer_copy(lla._QUERY.pack(1, 2, 3, 4, 5, 6, 7, 8, 9.0, *range(10, 16)))
    flat = [getattr(got, f[0]) for f in QueryStruct._fields_[:-1]] + list(got.reserved)
    assert flat == [1, 2, 3, 4, 5, 6, 7, 8, 9.0, *range(10, 16)]


@pytest.mark.parametrize("kw,status", [
    ({"d": 48}, UNSUPPORTED), ({"dv": 256}, UNSUPPORTED), ({"page_size": 8}, UNSUPPORTED),
    ({"page_size": 48}, UNSUPPORTED), ({"page_size": 2048}, UNSUPPORTED), ({"dtype": 2}, INVALID),
    ({"num_seqs": -1}, INVALID), ({"kv_heads": 0}, INVALID), ({"max_pages": -1}, INVALID),
    ({"num_pages": -1}, INVALID), ({"max_pages": 1 << 26}, UNSUPPORTED), ({"num_seqs": 65536}, UNSUPPORTED),
    ({"num_pages": 1 << 30}, UNSUPPORTED), ({"k_pages": None}, INVALID), ({"v_pages": 520}, INVALID),
    ({"page_table": None}, INVALID), ({"lens": None}, INVALID)])
def test_cache_refusals(lla, kw, status):
    c = cache(lla, **kw)
    lib = lla._load()
    assert attend(lla, c, query(lla)) == status
    assert lib.lla_paged_append(ctypes.byref(c), 256, 512, 768, 4, None) == status
    assert lib.lla_paged_evict(ctypes.byref(c), ctypes.byref(cache(lla, lens=4096, page_table=8192)), 4, 0, 0,
                               256, None) == (INVALID if status == OK else status) or status == UNSUPPORTED


@pytest.mark.parametrize("kw,status", [
    ({"q": None}, INVALID), ({"out": None}, INVALID), ({"q": 257}, INVALID), ({"r": 260}, INVALID),
    ({"starts": None}, INVALID), ({"tokens": -1}, INVALID), ({"max_new": -1}, INVALID), ({"max_new": 0}, INVALID),
    ({"q_heads": 3}, INVALID), ({"q_heads": 0}, INVALID), ({"h": 0.0}, INVALID), ({"h": float("nan")}, INVALID),
    ({"window": -1}, INVALID), ({"sinks": -1}, INVALID), ({"path": 3}, INVALID), ({"path": -1}, INVALID),
    ({"tokens": 1 << 30, "q_heads": 2}, UNSUPPORTED), ({"tokens": 0}, OK), ({"tokens": 0, "q": None}, OK)])
def test_query_refusals(lla, kw, status):
    assert attend(lla, cache(lla), query(lla, **kw)) == status


def test_reserved_fields_and_null_structs(lla):
    lib = lla._load()
    c, q = cache(lla), query(lla)
    q.reserved[0] = 1
    assert attend(lla, c, q) == INVALID
    c.reserved[1] = 1
    assert attend(lla, c, query(lla)) == INVALID
    assert lib.lla_paged_attention(None, ctypes.byref(query(lla)), None, 0, None) == INVALID
    assert lib.lla_paged_attention(ctypes.byref(cache(lla)), None, None, 0, None) == INVALID
    assert lib.lla_paged_append(None, 256, 256, 256, 1, None) == INVALID
    assert lib.lla_paged_evict(None, None, 1, 0, 0, 256, None) == INVALID


def test_tracking_needs_a_mass_and_scratch_its_size(lla):
    assert attend(lla, cache(lla, mass=None), query(lla, track_mass=1)) == INVALID
    big = cache(lla, max_pages=1024, num_pages=4096)
    need = lla._load().lla_paged_workspace_size(ctypes.byref(big), ctypes.byref(query(lla)))
    assert need > 0 and need % 256 == 0
    assert attend(lla, big, query(lla), 256, need - 1) == INVALID
    assert attend(lla, big, query(lla), 128, need) == INVALID
    assert lla._load().lla_paged_workspace_size(ctypes.byref(cache(lla, d=48)), ctypes.byref(query(lla))) == 0


def test_evict_refusals(lla):
    lib = lla._load()

    def call(frm={}, to={}, budget=8, sinks=0, recent=0, kept=256):
        a = cache(lla, **frm)
        b = cache(lla, **{"page_table": 8192, "lens": 4096, **to})
        return lib.lla_paged_evict(ctypes.byref(a), ctypes.byref(b), budget, sinks, recent, kept, None)
    assert call(budget=0) == INVALID
    assert call(sinks=-1) == INVALID and call(recent=-1) == INVALID
    assert call(sinks=5, recent=4) == INVALID
    assert call(sinks=2 ** 31 - 1, recent=2 ** 31 - 1) == INVALID
    assert call(kept=None) == INVALID
    assert call(to={"lens": 1280}) == INVALID and call(to={"page_table": 1024}) == INVALID
    assert call(to={"mass": None}) == INVALID and call(frm={"mass": None}) == INVALID
    assert call(to={"d": 32}) == INVALID and call(to={"num_seqs": 3}) == INVALID
    assert call(to={"page_size": 32}) == INVALID and call(to={"dtype": 0}) == INVALID
    assert call(budget=40, to={"max_pages": 2}) == INVALID    # 32 slots for 40 positions
    assert call(frm={"num_seqs": 0}, to={"num_seqs": 0}) == OK


def test_binding_checks(lla):
    meta = lambda *s, dtype=torch.bfloat16: torch.empty(*s, dtype=dtype)  # noqa: E731
    i32 = dict(dtype=torch.int32)
    good = dict(k_pages=meta(4, 2, 16, 64), v_pages=meta(4, 2, 16, 64), page_table=torch.zeros(1, 4, **i32),
                lens=torch.zeros(1, **i32))
    for bad in ({}, {"k_pages": meta(4, 2, 16)}, {"v_pages": meta(4, 2, 32, 64)},
                {"v_pages": meta(4, 2, 16, 64, dtype=torch.float32)},
                {"k_pages": meta(4, 2, 16, 64, dtype=torch.float16), "v_pages": meta(4, 2, 16, 64, dtype=torch.float16)},
                {"page_table": torch.zeros(1, 4)}, {"lens": torch.zeros(2, **i32)}, {"mass": torch.zeros(4, 2, 8)}):
        with pytest.raises(ValueError):  # {}: CPU tensors
            lla.PagedCache(**{**good, **bad})
