"""Host-side validation of the tree and cache calls: what memory and which scales they take.

CPU only: every call below has nothing to do or fails validation."""
import ctypes as C

import pytest

import draft_selection_amd as ds
import test_abi_tree as at

F = at.F


@pytest.fixture(scope="module")
def lib():
    return ds.lib()


def test_nothing_to_do_needs_no_memory(lib):
    """With no work every pointer may be NULL, those of the cache among them; its sizes are still checked."""
    for bad, code in ((dict(), 0), (dict(heads=0), -1), (dict(dim=100), -3), (dict(dt=0), -2), (dict(slot_stride=-8), -1)):
        c = at._cache(k=None, v=None, **bad)
        none = dict(q=None, out=None, page_table=None, seq_len=None, ws=None, wsb=0)
        assert at._attn(lib, c, batch=0, **none) == code
        for B, T in ((0, 9), (2, 0)):
            assert lib.dsel_cache_append(None, None, None, C.byref(c), None, 4, 4, None, B, T, None, None) == code
        assert lib.dsel_cache_compact(C.byref(c), None, 4, 4, None, None, None, 0, 9, None, None) == code
        p = ds.PagesArgs(None, 4, 0, 4, None, None, None, 10, 16)
        assert lib.dsel_pages_fork(C.byref(p), None, C.byref(c), None, None, 0, None) == code
    assert at._attn(lib, at._cache(k=None)) == -1 and at._attn(lib, at._cache(v=None)) == -1


def test_compact_writes_lengths_apart_from_what_it_reads(lib):
    """Workgroups of a row read its length, path and table while one of them writes new_len: no byte may be shared."""
    far = 1 << 20
    seq, path, n, table = F, F + far, F + 2 * far, F + 3 * far    # [5], [5, 9], [5], 5 rows of 4, 6 apart

    def compact(new):
        return lib.dsel_cache_compact(C.byref(at._cache(v=F + (1 << 30))), table, 6, 4, seq, path, n, 5, 9, new, None)
    for start, words in ((seq, 5), (n, 5), (path, 5 * 9), (table, 4 * 6 + 4)):
        for w in (-4, 0, words - 1):
            assert compact(start + 4 * w) == -1, (start, w)


@pytest.mark.parametrize("dt,size", [(1, 2), (2, 1)])
def test_writers_take_k_and_v_apart_or_as_one(lib, dt, size):
    """A V that begins inside K's first row, or the other way round, is refused by the calls that write the cache; so is
    one array as both for new rows, or scales, that are not the same for both."""
    page = ds.PagesArgs(F, 4, 2, 4, F, F, F, 10, 16)
    st = (C.c_int64 * 4)(0, 9 * 1024, 1024, 128)

    def append(c, v_new):
        return lib.dsel_cache_append(F, v_new, C.byref(st), C.byref(c), F, 4, 4, F, 2, 9, None, None)
    for shift in (16, 128 * size - 16, 16 - 128 * size):
        c = at._cache(dt=dt, v=F + shift)
        assert append(c, F) == -1 and append(c, F + 4096) == -1
        assert lib.dsel_cache_compact(C.byref(c), F, 4, 4, F, F, F, 2, 9, F + 4096, None) == -1
        assert lib.dsel_pages_fork(C.byref(page), F, C.byref(c), F, F, 1 << 20, None) == -1
    assert append(at._cache(dt=dt), F + 16) == -1
    if dt == 2:
        assert append(at._cache(dt=dt, k_scale=F, v_scale=F + 4), F) == -1


def test_scales_past_the_largest(lib):
    """Times log2(e) they are no finite fp32, and scores of 0 would become NaN."""
    for scale in (2.0 ** 127 * (1 + 2.0 ** -23), 3.4e38):
        assert at._attn(lib, scale=scale) == -1
