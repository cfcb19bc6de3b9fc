"""Host-side validation of the tree and cache calls: bad arguments are refused before anything is launched.

CPU only: every call below fails validation or has nothing to do."""
import ctypes as C
import inspect

import pytest
import torch

import draft_selection_amd as ds

F = 0x100000  # never dereferenced


@pytest.fixture(scope="module")
def lib():
    return ds.lib()


def _cache(**kw):
    a = dict(k=F, v=F, dt=1, layers=1, layer_stride=0, num_pages=10, page_stride=16 * 8 * 128, page_size=16,
             slot_stride=8 * 128, heads=8, head_stride=128, dim=128, k_scale=None, v_scale=None)
    a.update(kw)
    return ds.CacheArgs(*[a[n] for n, _ in ds.CacheArgs._fields_])


def _attn(lib, cache=None, ws=F, wsb=1 << 40, **kw):
    a = dict(q=F, q_batch=9 * 32 * 128, q_token=32 * 128, q_head=128, batch=2, block=9, q_heads=32, block_len=None,
             page_table=F, table_ld=4, max_pages=4, seq_len=F, mask=None, scale=0.1, out=F, lse=None)
    a.update(kw)
    return lib.dsel_tree_attn(C.byref(ds.TreeAttnArgs(*[a[n] for n, _ in ds.TreeAttnArgs._fields_])),
                              C.byref(cache or _cache()), ws, wsb, None)


BAD_CACHES = [
    (dict(k=None), -1), (dict(v=None), -1), (dict(dt=0), -2), (dict(dt=3), -2), (dict(layers=0), -1),
    (dict(layers=1025), -1), (dict(heads=0), -1), (dict(heads=1025), -1), (dict(dim=0), -1), (dict(dim=264), -1),
    (dict(dim=100), -3), (dict(num_pages=0), -1), (dict(num_pages=1 << 31), -1), (dict(page_size=0), -1),
    (dict(page_size=65537), -1), (dict(k=F + 8), -3), (dict(v=F + 2), -3), (dict(page_stride=64), -1),
    (dict(slot_stride=-1024), -1), (dict(head_stride=132), -3), (dict(page_stride=1 << 61), -1),
    (dict(k_scale=F), -1), (dict(dt=2, k_scale=F + 1), -3), (dict(dt=2, dim=72, head_stride=80), -3),
]


@pytest.mark.parametrize("kw,code", BAD_CACHES)
def test_cache_geometry_is_checked(lib, kw, code):
    c = _cache(**kw)
    if c.layers == 1:
        assert _attn(lib, c) == code
    st = (C.c_int64 * 4)(0, 9 * 1024, 1024, 128)
    assert lib.dsel_cache_append(F, F, C.byref(st), C.byref(c), F, 4, 4, F, 2, 9, None, None) == code
    assert lib.dsel_cache_compact(C.byref(c), F, 4, 4, F, F, F, 2, 9, F + 64, None) == code
    p = ds.PagesArgs(F, 4, 2, 4, F, F, F, 10, 16)
    assert lib.dsel_pages_fork(C.byref(p), F, C.byref(c), F, F, 1 << 20, None) == code


def test_tree_attn_validation(lib):
    assert lib.dsel_tree_attn(None, C.byref(_cache()), F, 1 << 40, None) == -1
    assert _attn(lib, _cache(layers=2, layer_stride=1 << 20)) == -1
    for kw in (dict(batch=-1), dict(batch=65536), dict(block=0), dict(block=257), dict(q_heads=0), dict(q_heads=12),
               dict(q_heads=2048), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")),
               dict(scale=float("inf")), dict(page_table=None), dict(seq_len=None), dict(max_pages=0),
               dict(table_ld=3), dict(max_pages=1 << 27, table_ld=1 << 27), dict(q=None), dict(out=None),
               dict(q_token=-8), dict(q_batch=1 << 60)):
        assert _attn(lib, **kw) == -1, kw
    for kw in (dict(q=F + 8), dict(out=F + 8), dict(lse=F + 2), dict(mask=F + 1), dict(q_head=132),
               dict(block_len=F + 2), dict(page_table=F + 2), dict(seq_len=F + 1)):
        assert _attn(lib, **kw) == -3, kw
    assert _attn(lib, batch=0, q=None, out=None, page_table=None, seq_len=None, ws=None, wsb=0) == 0
    need = lambda B=2, T=9, Hq=32, H=8, D=128, dt=1, n=1 << 20: lib.dsel_tree_attn_workspace_bytes(B, T, Hq, H, D, dt, n)
    assert need() > 0 and need(n=64) == 0 and need(T=257) == 0 and need(Hq=12) == 0 and need(dt=0) == 0 and need(D=257) == 0
    wide = dict(table_ld=1 << 16, max_pages=1 << 16)
    assert _attn(lib, wsb=need() - 1, **wide) == -4 and _attn(lib, ws=None, **wide) == -4
    assert _attn(lib, ws=F + 8, **wide) == -3


def test_tree_mask_and_accept_validation(lib):
    m = lambda parent=F, B=2, T=9, lens=None, mask=F, depth=F: lib.dsel_tree_mask(parent, B, T, lens, mask, depth, None)
    assert m(T=0) == -1 and m(T=257) == -1 and m(B=-1) == -1 and m(parent=None) == -1 and m(mask=None) == -1
    assert m(parent=F + 2) == -3 and m(lens=F + 2) == -3 and m(depth=F + 1) == -3
    assert m(B=0, parent=None, mask=None) == 0
    a = dict(parent=F, tok=F, target=F, step=1, B=2, T=9, lens=None, n=F, path=F, out=F)
    call = lambda **kw: lib.dsel_tree_accept(*{**a, **kw}.values(), None)
    assert call(T=257) == -1 and call(step=0) == -1 and call(step=1 << 31) == -1
    for k in ("parent", "tok", "target", "n", "path", "out"):
        assert call(**{k: None}) == -1 and call(**{k: F + 2}) == -3
    assert call(B=0, parent=None, tok=None) == 0


def test_append_and_compact_validation(lib):
    def append(k=F, v=F, st=(0, 9 * 1024, 1024, 128), table=F, ld=4, n=4, seq=F, B=2, T=9, lens=None):
        return lib.dsel_cache_append(k, v, (C.c_int64 * 4)(*st) if st else None, C.byref(_cache()), table, ld, n, seq, B,
                                     T, lens, None)
    assert append(k=None) == -1 and append(v=None) == -1 and append(st=None) == -1 and append(T=-1) == -1
    assert append(st=(0, 9 * 1024, 1020, 128)) == -3 and append(st=(0, -8, 1024, 128)) == -1 and append(k=F + 4) == -3
    assert append(table=None) == -1 and append(seq=None) == -1 and append(ld=2) == -1 and append(lens=F + 1) == -3
    assert append(B=0, k=None, v=None) == 0 and append(T=0, k=None, v=None) == 0 and append(B=65536) == -1
    # one token past the longest block: a grid of 2^32 threads comes at twice that, and no device takes it
    assert append(st=(0, 0, 0, 128), T=(1 << 29) + 1) == -1 and append(st=(0, 0, 0, 128), T=(1 << 30) - 1) == -1

    def compact(table=F, seq=F, path=F, n=F, B=2, T=9, new=F + 64):
        return lib.dsel_cache_compact(C.byref(_cache()), table, 4, 4, seq, path, n, B, T, new, None)
    assert compact(path=None) == -1 and compact(n=None) == -1 and compact(new=None) == -1
    assert compact(new=F) == -1                      # the lengths that other workgroups still read
    assert compact(path=F + 2) == -3 and compact(T=0) == -1 and compact(T=257) == -1
    assert compact(B=0, table=None, path=None) == 0


def test_pages_validation(lib):
    def pages(**kw):
        a = dict(table=F, ld=4, rows=3, max_pages=4, row_pages=F, seq_len=F, refcount=F, num_pages=10, page_size=16)
        a.update(kw)
        return ds.PagesArgs(*a.values())
    calls = [lambda p, arg=F, g=F: lib.dsel_pages_reserve(C.byref(p), arg, g, None),
             lambda p, arg=F, g=F: lib.dsel_pages_fork(C.byref(p), arg, C.byref(_cache()), g, F, 1 << 20, None),
             lambda p, arg=F, g=F: lib.dsel_pages_free(C.byref(p), arg, None)]
    for i, f in enumerate(calls):
        for kw in (dict(rows=-1), dict(rows=4097), dict(max_pages=0), dict(ld=3), dict(num_pages=0),
                   dict(page_size=0), dict(page_size=65537), dict(table=None), dict(row_pages=None),
                   dict(seq_len=None), dict(refcount=None), dict(max_pages=1 << 28, ld=1 << 28)):
            assert f(pages(**kw)) == -1, kw
        for k in ("table", "row_pages", "seq_len", "refcount"):
            assert f(pages(**{k: F + 2})) == -3
        assert f(pages(), arg=None) == -1 and f(pages(), arg=F + 2) == -3
        assert f(pages(rows=0, table=None), arg=None) == 0
        if i < 2:
            assert f(pages(), g=None) == -1 and f(pages(), g=F + 1) == -3
    assert lib.dsel_pages_reserve(None, F, F, None) == -1 and lib.dsel_pages_free(None, F, None) == -1
    fork = lambda p=pages(), c=_cache(), ws=F, b=1 << 20: lib.dsel_pages_fork(C.byref(p), F, C.byref(c), F, ws, b, None)
    assert fork(pages(num_pages=11)) == -1 and fork(pages(page_size=32)) == -1    # not the cache's
    assert fork(ws=None) == -4 and fork(b=11) == -4 and fork(ws=F + 2) == -3
    assert lib.dsel_pages_fork_workspace_bytes(3) == 12 and lib.dsel_pages_fork_workspace_bytes(4097) == 0


def test_binding_refuses_host_tensors():
    import torch

    z = torch.zeros((2, 3), dtype=torch.int32)
    for f, args in ((ds.tree_mask, (z,)), (ds.tree_accept, (z, z, z)),
                    (ds.pages_free, (ds.Pages(z, z[:, 0], z[:, 0], z[0], 16), z[:, 0]))):
        with pytest.raises(ValueError):
            f(*args)


def test_calls_take_their_arguments_by_name():
    """The first argument, whose device a call runs on, may be given by name as any other; a missing one is named."""
    x = torch.zeros(2, 3, dtype=torch.int32)
    pages = ds.Pages(x, x[:, 0], x[:, 0], x[0], 16)
    for fn, kw in [(ds.tree_mask, dict(parent=x)), (ds.tree_accept, dict(parent=x, tok=x, target_tok=x)),
                   (ds.tree_attn, dict(q=x, k_cache=x, v_cache=x, page_table=x, seq_len=x)),
                   (ds.cache_append, dict(k_new=x, v_new=x, k_cache=x, v_cache=x, page_table=x, seq_len=x)),
                   (ds.cache_compact, dict(k_cache=x, v_cache=x, page_table=x, seq_len=x, path=x, n_keep=x)),
                   (ds.pages_reserve, dict(pages=pages, extra=x)), (ds.pages_free, dict(pages=pages, which=x)),
                   (ds.pages_fork, dict(pages=pages, src=x, k_cache=x, v_cache=x))]:
        with pytest.raises(ValueError, match="on the GPU"):
            fn(**kw)
        with pytest.raises(TypeError, match="missing"):
            fn()
        assert list(inspect.signature(fn).parameters)[-1] == "stream"
