"""Host-side checks of the page operators: refusals before any HIP call; and the tests' own reference."""
import ctypes
import os

import pytest
import torch

import device_wide_prefix_amd as dws
from pages_reference import Cache, filled, pages_of

FAKE = 0x100000      # never dereferenced
BAD, UNSUPPORTED, OVERLAP, MISALIGNED = dws.ERR_INVALID_ARG, dws.ERR_UNSUPPORTED, dws.ERR_OVERLAP, dws.ERR_MISALIGNED


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(dws.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    return dws.load_library()


def cache(**more):
    return dws.PageCache(**{"d_refs": FAKE, "n_pages": 100, "d_table": FAKE + 0x1000, "n_rows": 10, "max_pages": 20,
                            "d_lengths": FAKE + 0x2000, "page_tokens": 16, **more})


def room(k):
    return FAKE + 0x10000 * k


CALLS = {
    "grow": lambda lib, c, n, a, w, size: lib.dws_pages_grow(c, a, room(2), n, room(3), w, size, None),
    "fork": lambda lib, c, n, a, w, size: lib.dws_pages_fork(c, a, room(2), n, room(3), room(4), room(5), room(6), w, size, None),
    "free": lambda lib, c, n, a, w, size: lib.dws_pages_free(c, a, n, room(6), w, size, None),
}


@pytest.mark.parametrize("name", list(CALLS))
def test_refusals(lib, name):
    def call(c, n=5, a=room(1), w=room(9), size=1 << 20):
        return CALLS[name](lib, None if c is None else ctypes.byref(c), n, a, w, size)

    assert call(None) == BAD
    for more, status in (({"d_refs": None}, BAD), ({"n_pages": 0}, BAD), ({"n_pages": -5}, BAD), ({"n_rows": -1}, BAD),
                         ({"max_pages": -1}, BAD), ({"page_tokens": 0}, BAD), ({"d_table": None}, BAD),
                         ({"d_lengths": None}, BAD), ({"n_pages": (1 << 24) + 1}, UNSUPPORTED),
                         ({"page_tokens": 1 << 31}, UNSUPPORTED), ({"n_rows": 1 << 31}, UNSUPPORTED),
                         ({"n_rows": 1 << 30, "max_pages": 1 << 30}, UNSUPPORTED), ({"d_refs": FAKE + 2}, MISALIGNED),
                         ({"d_lengths": FAKE + 0x1010}, OVERLAP), ({"d_table": FAKE + 0x10}, OVERLAP)):
        assert call(cache(**more)) == status, more
    assert call(cache(), n=-1) == BAD
    assert call(cache(max_pages=1 << 20), n=1 << 30) == UNSUPPORTED
    assert call(cache(), a=None) == BAD
    assert call(cache(), a=room(1) + 1) == MISALIGNED
    assert call(cache(), a=FAKE + 4) == OVERLAP
    assert call(cache(), w=None) == BAD
    assert call(cache(), size=16) == BAD
    assert call(cache(), w=room(9) + 64) == MISALIGNED
    assert call(cache(), w=FAKE) == OVERLAP


def test_refusals_of_compact_and_workspace(lib):
    def call(c, remap=room(1), src=room(2), dst=room(3), moves=room(4), count=room(5), w=room(9), size=1 << 20):
        return lib.dws_pages_compact(ctypes.byref(c), remap, src, dst, moves, count, w, size, None)

    for more in ({"remap": None}, {"src": None}, {"dst": None}, {"moves": None}, {"count": None}, {"w": None}, {"size": 0}):
        assert call(cache(), **more) == BAD, more
    assert call(cache(), count=room(5) + 4) == MISALIGNED
    assert call(cache(), dst=room(2) + 8) == OVERLAP
    assert call(cache(), count=room(4)) == OVERLAP
    assert call(cache(n_pages=0)) == BAD
    need = ctypes.c_size_t(0)
    size = lib.dws_pages_workspace
    assert size(None, 0, ctypes.byref(need)) == BAD and size(ctypes.byref(cache()), 0, None) == BAD
    assert size(ctypes.byref(cache()), -1, ctypes.byref(need)) == BAD
    assert size(ctypes.byref(cache(n_pages=1 << 25)), 1, ctypes.byref(need)) == UNSUPPORTED
    assert size(ctypes.byref(cache()), 5, ctypes.byref(need)) == dws.OK and need.value >= 4 * (100 + 10 + 2 * 5 + 1)


def test_refusals_of_copy(lib):
    def call(pool=FAKE, pages=10, page=64, layers=2, stride=640, src=room(1), dst=room(2), n=3, count=None):
        return lib.dws_pages_copy(pool, pages, page, layers, stride, src, dst, n, count, None)

    for more in ({"pool": None}, {"pages": -1}, {"page": -1}, {"layers": -1}, {"stride": 639}, {"stride": -1}, {"src": None},
                 {"dst": None}, {"n": -1}, {"pool": 2**64 - 64}):
        assert call(**more) == BAD, more
    for more in ({"pages": 1 << 31}, {"page": 1 << 51}, {"layers": 1 << 31}, {"pages": 1 << 30, "page": 1 << 30, "stride": 1 << 49},
                 {"n": 1 << 31}):
        assert call(**more) == UNSUPPORTED, more
    assert call(src=room(1) + 2) == MISALIGNED and call(count=room(3) + 4) == MISALIGNED
    assert call(src=FAKE + 64) == OVERLAP and call(count=FAKE + 8) == OVERLAP
    for more in ({"n": 0}, {"pages": 0}, {"page": 0}, {"layers": 0}):
        assert call(**{"pool": None, "src": None, "dst": None, **more}) == dws.OK, more


def test_packed_cache_is_the_structure():
    values = [FAKE + 8 * i for i in range(7)]
    c = dws.PageCache(*values)
    assert dws._PAGES.size == ctypes.sizeof(c) and dws._PAGES.pack(*values) == bytes(c)


def test_binding_refuses_cpu_tensors():
    x = torch.zeros(4, dtype=torch.int32)
    table = torch.zeros(2, 2, dtype=torch.int32)
    for call in (lambda: dws.pages_grow(x, table, x[:2], x, x, 1), lambda: dws.pages_fork(x, table, x[:2], x, x, 1),
                 lambda: dws.pages_free(x, table, x[:2], x, 1), lambda: dws.pages_compact(x, table),
                 lambda: dws.pages_copy(x, x, x)):
        with pytest.raises(TypeError):
            call()


@pytest.mark.parametrize("seed", range(5))
def test_reference_keeps_its_books(seed):
    """Counts are the entries that name a page, and rows hold as many pages as their lengths need."""
    c = filled(seed, 60, 9, 8, 4)

    def books():
        held = [0] * 60
        for row, n in zip(c.table, c.lengths):
            pages = row[: pages_of(n, 4)]
            assert all(p >= 0 for p in pages) and all(p == -1 for p in row[len(pages):])
            for p in pages:
                held[p] += 1
        assert held == c.refs

    books()
    count = c.compact()[0]
    assert all(n > 0 for n in c.refs[:count]) and not any(c.refs[count:])
    books()
    c.free(range(9))
    books()
    assert c.refs == [0] * 60 and Cache(60, 9, 8, 4).refs == c.refs
