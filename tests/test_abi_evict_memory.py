"""cache_evict's arguments on top of each other: refused on the host, before anything is launched.

CPU only: every call below is refused."""
import ctypes as C
import itertools

import pytest

import draft_selection_amd as ds
import test_abi_tree as at

F = at.F
ROWS, PAGES, P, N = 3, 4, 16, 10
LD = 80                                   # weights' and kept's rows: 64 positions and a gap of 16
BYTES = dict(weights=(ROWS - 1) * LD * 4 + 256, kept=(ROWS - 1) * LD * 4 + 256, budget=12, granted=4, ws=2 * 16 + 48 + 2 * 768,
             table=(ROWS - 1) * 24 + 16, row_pages=12, seq_len=12, refcount=N * 4)


@pytest.fixture(scope="module")
def lib():
    return ds.lib()


def _evict(lib, **where):
    a = {n: F + (i + 1) * (1 << 16) for i, n in enumerate(BYTES)}
    a.update(where)
    pages = ds.PagesArgs(a["table"], 6, ROWS, PAGES, a["row_pages"], a["seq_len"], a["refcount"], N, P)
    return lib.dsel_cache_evict(C.byref(pages), a["budget"], a["weights"], LD, 0, 0, C.byref(at._cache(v=F + (1 << 30))), a["kept"],
                                a["granted"], a["ws"], BYTES["ws"], None)


WRITTEN = ["weights", "kept", "budget", "granted", "ws"]
PAIRS = [(x, y) for x, y in itertools.product(WRITTEN, BYTES) if x != y]


@pytest.mark.parametrize("x,y", PAIRS)
def test_nothing_lies_on_anything_else(lib, x, y):
    base = F + (1 << 28)
    step = 16 if "ws" in (x, y) else 4
    assert _evict(lib, **{x: base, y: base}) == -1
    # the last bytes of y under the first of x
    last = (BYTES[y] - 1) // step * step
    assert _evict(lib, **{x: base + last, y: base}) == -1, (x, y)


def test_rows_that_reach_into_each_other(lib):
    """Rows of 64 in steps of 80: another array's rows do not fit between them, a few values would."""
    base = F + (1 << 28)
    for off in (4, 63 * 4, 65 * 4, 79 * 4, LD * 4, LD * 4 + 60, 2 * LD * 4):
        assert _evict(lib, weights=base, kept=base + off) == -1, off
        assert _evict(lib, weights=base + off, kept=base) == -1, off
    for off in (62 * 4, LD * 4 - 4, LD * 4 + 63 * 4, 2 * LD * 4 + 63 * 4):
        assert _evict(lib, weights=base, budget=base + off) == -1, off
        assert _evict(lib, kept=base, seq_len=base + off) == -1, off
    # a table whose rows (16 bytes of 24) run through the gap into the second row
    assert _evict(lib, weights=base, table=base + LD * 4 - 40) == -1
    assert _evict(lib, weights=base, table=base + 250) == -3 and _evict(lib, weights=base, table=base + 252) == -1
