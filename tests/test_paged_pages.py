"""The refusals of fork, free, grow, copy and compact, on the CPU (decided on the host; pointers are never
dereferenced), and which device and stream the binding's calls run on."""
import ctypes

import pytest
import torch

from test_paged_abi import INVALID, OK, UNSUPPORTED, cache, lla  # noqa: F401
from test_paged_binding import Fake, Machine, binding, calls, problem  # noqa: F401


def byref(lla, kw):  # noqa: F811
    return ctypes.byref(cache(lla, **kw))


BAD_CACHES = [(dict(d=48), UNSUPPORTED), (dict(page_size=48), UNSUPPORTED), (dict(dtype=2), INVALID),
              (dict(k_pages=None), INVALID), (dict(page_table=None), INVALID), (dict(lens=None), INVALID)]


def test_fork(lla):  # noqa: F811
    def call(frm={}, to={}, parents=256, refs=512):
        return lla._load().lla_paged_fork(byref(lla, frm), byref(lla, {"page_table": 8192, "lens": 4096, **to}), parents,
                                          refs, None)
    for kw, status in BAD_CACHES:
        assert call(frm=kw) == status and call(to=kw) == status
    assert call(parents=None) == INVALID and call(refs=None) == INVALID and call(refs=516) == INVALID
    assert call(to={"lens": 1280}) == INVALID and call(to={"page_table": 1024}) == INVALID
    for kw in ({"k_pages": 4096}, {"v_pages": 4096}, {"num_pages": 21}, {"kv_heads": 1}, {"page_size": 32}, {"dv": 32}):
        assert call(to=kw) == INVALID
    assert call(to={"num_seqs": 0}) == OK


def test_free_and_grow(lla):  # noqa: F811
    lib = lla._load()
    free = lambda refs=512, **kw: lib.lla_paged_free(byref(lla, kw), None, refs, None)  # noqa: E731

    def grow(starts=256, refs=512, copies=1024, left=2048, **kw):
        return lib.lla_paged_grow(byref(lla, kw), starts, refs, copies, left, None)
    for kw, status in BAD_CACHES:
        assert free(**kw) == status and grow(**kw) == status
    assert free(refs=None) == INVALID and free(refs=514) == INVALID and free(num_seqs=0) == OK
    for name in ("starts", "refs", "copies", "left"):
        assert grow(**{name: None}) == INVALID
    assert grow(refs=516) == INVALID and grow(copies=1028) == INVALID
    assert grow(num_seqs=4097) == UNSUPPORTED


def test_copy(lla):  # noqa: F811
    def call(frm={}, to={}, pairs=256, count=3):
        return lla._load().lla_paged_copy(byref(lla, frm), byref(lla, to), pairs, count, None)
    for kw, status in BAD_CACHES[:4]:
        assert call(frm=kw) == status and call(to=kw) == status
    for kw in ({"kv_heads": 1}, {"page_size": 32}, {"dv": 32}, {"dtype": 0}, {"v_pages": 520}, {"mass": 772}):
        assert call(to=kw) == INVALID
    assert call(pairs=None) == INVALID and call(pairs=260) == INVALID and call(count=-1) == INVALID
    assert call(count=0) == OK and call(count=0, pairs=None) == OK


def test_compact(lla):  # noqa: F811
    def call(starts=256, tokens=4, path=512, max_path=2, keep=1024, **kw):
        return lla._load().lla_paged_compact(byref(lla, kw), starts, tokens, path, max_path, keep, None)
    for kw, status in BAD_CACHES:
        assert call(**kw) == status
    for name in ("starts", "path", "keep"):
        assert call(**{name: None}) == INVALID
    assert call(tokens=-1) == INVALID and call(max_path=-1) == INVALID and call(tokens=1 << 30) == UNSUPPORTED
    assert call(num_seqs=0) == OK


def test_tree_attention(lla):  # noqa: F811
    from test_paged_abi import query
    lib = lla._load()

    def call(parents=256, c={}, **kw):
        q = query(lla, **kw)
        return lib.lla_paged_tree_attention(byref(lla, c), ctypes.byref(q), parents, None, 0, None)
    for kw, status in BAD_CACHES:
        assert call(c=kw) == status
    assert call(parents=None) == INVALID and call(track_mass=1) == INVALID and call(max_new=0) == INVALID
    assert call(tokens=2000, max_new=1025) == UNSUPPORTED and call(tokens=0, max_new=5000, parents=None) == OK
    size = lambda **kw: lib.lla_paged_tree_workspace_size(byref(lla, {}), ctypes.byref(query(lla, **kw)))  # noqa: E731
    plain = lib.lla_paged_workspace_size(byref(lla, {}), ctypes.byref(query(lla, tokens=600, max_new=300)))
    assert size(tokens=600, max_new=300) >= plain + 600 * 44  # ten words of bits and a depth for each node
    assert size(tokens=2000, max_new=1025) == 0 and size(track_mass=1) == 0


@pytest.mark.parametrize("index", [0, 1])
def test_calls_run_on_the_device_of_the_cache(calls, index):  # noqa: F811
    cache_, to, rows, starts, out, lse = problem(index)
    i32 = lambda *s: Fake(*s, dtype=torch.int32, index=index)  # noqa: E731
    spec = binding.RotarySpec(64, freq=[1.0] * 32)
    binding.lla_paged_append_rotary(rows, rows, cache_, starts, spec, rows, q_out=rows)
    binding.lla_paged_tree_attention(rows, cache_, starts, i32(5), 8.0, out=out, lse=lse)
    binding.lla_paged_fork(cache_, to, i32(3), i32(4))
    binding.lla_paged_free(cache_, i32(4), i32(3))
    binding.lla_paged_grow(cache_, starts, i32(4), i32(3, 2), i32(1))
    binding.lla_paged_copy(cache_, to, i32(7, 2))
    binding.lla_paged_compact(cache_, starts, i32(3, 2), keep=i32(3))
    names = ("append_rotary", "tree_attention", "fork", "free", "grow", "copy", "compact")
    assert calls == [(f"lla_paged_{x}", index, 100 + index) for x in names] and Machine.current == 0


def test_tensors_of_another_kind_or_place_are_refused(calls):  # noqa: F811
    cache_, to, rows, starts, out, lse = problem(1)
    i32 = lambda *s, index=1, **kw: Fake(*s, dtype=torch.int32, index=index, **kw)  # noqa: E731
    spec = binding.RotarySpec(64, freq=[1.0] * 32)
    bad = [lambda: binding.lla_paged_fork(cache_, to, i32(2), i32(4)), lambda: binding.lla_paged_fork(cache_, to, i32(3), i32(5)),
           lambda: binding.lla_paged_fork(cache_, problem(0)[0], i32(3), i32(4)),
           lambda: binding.lla_paged_free(cache_, i32(4, index=0)), lambda: binding.lla_paged_free(cache_, i32(4), i32(2)),
           lambda: binding.lla_paged_grow(cache_, starts, i32(4), i32(3)), lambda: binding.lla_paged_grow(cache_, starts, i32(3)),
           lambda: binding.lla_paged_grow(cache_, starts, i32(4), i32(3, 2), i32(2)),
           lambda: binding.lla_paged_copy(cache_, to, i32(7, 3)),
           lambda: binding.lla_paged_copy(cache_, to, i32(7, 2, contiguous=False)),
           lambda: binding.lla_paged_compact(cache_, starts, i32(3), keep=i32(3)),
           lambda: binding.lla_paged_compact(cache_, starts, i32(2, 2), keep=i32(3)),
           lambda: binding.lla_paged_compact(cache_, starts, i32(3, 2), keep=i32(4)),
           lambda: binding.lla_paged_tree_attention(rows, cache_, starts, i32(4), 8.0, out=out, lse=lse),
           lambda: binding.lla_paged_append_rotary(rows, rows, cache_, starts, spec, None, r=rows),
           lambda: binding.lla_paged_append_rotary(rows, rows, cache_, starts, spec, rows, offsets=i32(4)),
           lambda: binding.lla_paged_append_rotary(rows, rows, cache_, starts, spec, rows, q_out=Fake(5, 3, 64))]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    assert not calls


def test_compact_does_not_write_the_lengths_it_reads(lla):  # noqa: F811
    assert lla._load().lla_paged_compact(byref(lla, {}), 256, 4, 512, 2, 1280, None) == INVALID


@pytest.mark.gpu
def test_copy_beyond_the_grid(lla):  # noqa: F811
    """2^30 pairs of pages of 512 KB: refused before a launch, with the device asked for its status word alone."""
    big = byref(lla, dict(page_size=1024, kv_heads=2, d=64, dv=64))
    assert lla._load().lla_paged_copy(big, big, 256, 1 << 30, None) == UNSUPPORTED
