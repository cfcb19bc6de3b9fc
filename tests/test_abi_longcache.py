"""Host-side validation of the long caches' calls, and the refusals of their binding.

CPU only: every call below fails validation or has nothing to do."""
import ctypes as C
import inspect

import pytest
import torch

import draft_selection_amd as ds
import test_abi_tree as at

F = at.F


@pytest.fixture(scope="module")
def lib():
    return ds.lib()


def _fp4(**kw):
    return at._cache(**{**dict(dt=4, k_scale=F + (1 << 30), v_scale=F + (2 << 30), v=F + (3 << 30)), **kw})


def _window(lib, window=64, sinks=4, depth=None, cache=None, ws=F, wsb=1 << 40, **kw):
    a = dict(q=F, q_batch=9 * 32 * 128, q_token=32 * 128, q_head=128, batch=2, block=9, q_heads=32, block_len=None,
             page_table=F, table_ld=4, max_pages=4, seq_len=F, mask=None, scale=0.1, out=F, lse=None)
    a.update(kw)
    return lib.dsel_tree_attn_window(C.byref(ds.TreeAttnArgs(*[a[n] for n, _ in ds.TreeAttnArgs._fields_])),
                                     C.byref(cache or at._cache()), window, sinks, depth, ws, wsb, None)


def _weights(lib, count=None, decay=1.0, w=F + (1 << 24), ld=64, cache=None, **kw):
    a = dict(q=F, q_batch=9 * 32 * 128, q_token=32 * 128, q_head=128, batch=2, block=9, q_heads=32, block_len=None,
             page_table=F, table_ld=4, max_pages=4, seq_len=F, mask=None, scale=0.1, out=None, lse=F)
    a.update(kw)
    return lib.dsel_key_weights(C.byref(ds.TreeAttnArgs(*[a[n] for n, _ in ds.TreeAttnArgs._fields_])),
                                C.byref(cache or at._cache()), count, decay, w, ld, None)


BAD_4BIT = [
    (dict(k_scale=None), -1), (dict(v_scale=None), -1), (dict(dim=80), -3), (dict(dim=16), -3), (dict(dim=288), -1),
    (dict(head_stride=144), -3), (dict(head_stride=96), -1), (dict(slot_stride=8 * 128 + 16), -3), (dict(k=F + 8), -3),
    (dict(k=None), -1), (dict(dt=3), -2), (dict(dt=5), -2),
]


@pytest.mark.parametrize("kw,code", BAD_4BIT)
def test_four_bit_caches_are_checked(lib, kw, code):
    c = _fp4(**kw)
    st = (C.c_int64 * 4)(0, 9 * 1024, 1024, 128)
    p = ds.PagesArgs(F, 4, 2, 4, F, F, F, 10, 16)
    assert at._attn(lib, c) == code and _window(lib, cache=c) == code
    assert lib.dsel_cache_append(F, F, C.byref(st), C.byref(c), F, 4, 4, F, 2, 9, None, None) == code
    assert lib.dsel_cache_compact(C.byref(c), F, 4, 4, F, F, F, 2, 9, F + 64, None) == code
    assert lib.dsel_pages_fork(C.byref(p), F, C.byref(c), F, F, 1 << 20, None) == code
    assert lib.dsel_cache_evict(C.byref(p), F, F, 64, 0, 0, C.byref(c), None, F, F, 1 << 20, None) == code
    if "v_scale" not in kw:
        assert _weights(lib, cache=c) == code


def test_four_bit_scales_go_with_their_rows(lib):
    """One array as K and V has one array of scales; of two, the scales are apart too."""
    st = (C.c_int64 * 4)(0, 9 * 1024, 1024, 128)
    p = ds.PagesArgs(F, 4, 2, 4, F, F, F, 10, 16)
    for c in (_fp4(v=F), _fp4(v=F + 16), _fp4(v_scale=F + (1 << 30)), _fp4(v_scale=F + (1 << 30) + 3)):
        assert lib.dsel_cache_append(F, F, C.byref(st), C.byref(c), F, 4, 4, F, 2, 9, None, None) == -1
        assert lib.dsel_cache_compact(C.byref(c), F, 4, 4, F, F, F, 2, 9, F + 64, None) == -1
        assert lib.dsel_pages_fork(C.byref(p), F, C.byref(c), F, F, 1 << 20, None) == -1
        assert lib.dsel_cache_evict(C.byref(p), F, F, 64, 0, 0, C.byref(c), None, F, F, 1 << 20, None) == -1


def test_window_validation(lib):
    assert lib.dsel_tree_attn_window(None, C.byref(at._cache()), 1, 0, None, F, 1 << 40, None) == -1
    assert _window(lib, window=0) == -1 and _window(lib, window=-5) == -1 and _window(lib, sinks=-1) == -1
    assert _window(lib, depth=F + 2) == -3 and _window(lib, mask=F + 1) == -3 and _window(lib, q=F + 8) == -3
    assert _window(lib, scale=0.0) == -1 and _window(lib, q_heads=12) == -1 and _window(lib, out=None) == -1
    none = dict(q=None, out=None, page_table=None, seq_len=None, ws=None, wsb=0)
    assert _window(lib, batch=0, **none) == 0 and _window(lib, batch=0, window=0, **none) == -1
    need = lambda B=2, T=9, Hq=32, H=8, D=128, dt=1, n=1 << 20, w=4096, s=4: \
        lib.dsel_tree_attn_window_workspace_bytes(B, T, Hq, H, D, dt, n, w, s)
    assert need() > 0 and need(w=50) == 0 and need(n=64) == 0 and need(w=0) == 0 and need(s=-1) == 0 and need(dt=3) == 0
    assert need(w=1 << 62, s=1 << 62) == need(w=1 << 20) > 0 and need(w=100, s=1 << 62) > 0 and need(dt=4) > 0
    wide = dict(table_ld=1 << 16, max_pages=1 << 16, window=4096)
    assert _window(lib, wsb=need() - 1, **wide) == -4 and _window(lib, ws=None, **wide) == -4
    assert _window(lib, ws=F + 8, **wide) == -3


def test_key_weights_validation(lib):
    for kw in (dict(decay=-0.1), dict(decay=1.5), dict(decay=float("nan")), dict(ld=63), dict(ld=1 << 61), dict(w=None),
               dict(lse=None), dict(q=None), dict(batch=-1), dict(block=257), dict(q_heads=12), dict(scale=-1.0),
               dict(page_table=None), dict(seq_len=None), dict(q_token=-8),
               # weights on top of what is read
               dict(w=F), dict(lse=F + (1 << 24)), dict(count=F + (1 << 24) + 4), dict(page_table=F + (1 << 24) + 64),
               dict(block_len=F + (1 << 24))):
        assert _weights(lib, **kw) == -1, kw
    for kw in (dict(w=F + 2), dict(count=F + 1), dict(lse=F + 2), dict(q=F + 8), dict(q_head=132), dict(seq_len=F + 1)):
        assert _weights(lib, **kw) == -3, kw
    assert _weights(lib, cache=at._cache(layers=2, layer_stride=1 << 20)) == -1
    assert lib.dsel_key_weights(None, C.byref(at._cache()), None, 1.0, F, 64, None) == -1
    a = ds.TreeAttnArgs(batch=2, block=9, q_heads=32)
    assert lib.dsel_key_weights(C.byref(a), None, None, 1.0, F, 64, None) == -1
    assert _weights(lib, batch=0, q=None, lse=None, w=None, page_table=None, seq_len=None) == 0
    # V is not looked at
    assert _weights(lib, batch=0, cache=at._cache(v=None)) == 0


def test_evict_validation(lib):
    def evict(budget=F, w=F, ld=64, sinks=0, recent=0, c=None, kept=None, g=F, ws=F, b=1 << 20, **kw):
        a = dict(table=F, ld=4, rows=3, max_pages=4, row_pages=F, seq_len=F, refcount=F, num_pages=10, page_size=16)
        a.update(kw)
        return lib.dsel_cache_evict(C.byref(ds.PagesArgs(*a.values())), budget, w, ld, sinks, recent,
                                    C.byref(c or at._cache(v=F + (1 << 30))), kept, g, ws, b, None)
    for kw in (dict(budget=None), dict(w=None), dict(g=None), dict(ld=63), dict(sinks=-1), dict(recent=-1), dict(rows=4097),
               dict(num_pages=11), dict(page_size=32), dict(table=None), dict(max_pages=5)):
        assert evict(**kw) == -1, kw
    for kw in (dict(budget=F + 2), dict(w=F + 2), dict(g=F + 1), dict(kept=F + 1), dict(ws=F + 8), dict(refcount=F + 2)):
        assert evict(**kw) == -3, kw
    need = lib.dsel_cache_evict_workspace_bytes(3, 64, 16)
    assert need == 2 * 16 + 48 + 2 * 768
    assert evict(ws=None) == -4 and evict(b=need - 1) == -4
    assert evict(rows=0, table=None, budget=None, w=None, g=None, ws=None, b=0) == 0
    for bad in ((0, 64, 16), (4097, 64, 16), (3, 60, 16), (3, 0, 16), (3, 64, 0), (3, 1 << 31, 16)):
        assert lib.dsel_cache_evict_workspace_bytes(*bad) == 0
    assert lib.dsel_cache_evict(None, F, F, 64, 0, 0, C.byref(at._cache()), None, F, F, 1 << 20, None) == -1


def test_calls_take_their_arguments_by_name():
    x = torch.zeros(2, 3, dtype=torch.int32)
    pages = ds.Pages(x, x[:, 0], x[:, 0], x[0], 16)
    for fn, kw in [(ds.tree_attn_window, dict(q=x, k_cache=x, v_cache=x, page_table=x, seq_len=x, window=3)),
                   (ds.key_weights, dict(q=x, lse=x, k_cache=x, page_table=x, seq_len=x, weights=x)),
                   (ds.cache_evict, dict(pages=pages, budget=x, weights=x, k_cache=x, v_cache=x))]:
        with pytest.raises(ValueError, match="on the GPU"):
            fn(**kw)
        with pytest.raises(TypeError, match="missing"):
            fn()
        assert list(inspect.signature(fn).parameters)[-1] == "stream"


def _pack4(P=16, H=2, D=64, s=lambda t: t, k=lambda t: t, k_dt=torch.float4_e2m1fn_x2, s_dt=torch.float8_e8m0fnu):
    kc = k(torch.zeros((3, P, H, D // 2), dtype=torch.uint8)).view(k_dt)
    sc = s(torch.zeros((3, P, H, D // 32), dtype=torch.uint8)).view(s_dt)
    return ds._cache(kc.device, kc, kc, sc, sc)


def test_binding_checks_the_scales_of_four_bit_caches():
    packed, shape = _pack4()
    assert shape == (1, 3, 16, 2, 64) and len(packed) == C.sizeof(ds.CacheArgs)
    c = ds.CacheArgs.from_buffer_copy(packed)
    assert (c.dt, c.dim, c.head_stride, c.slot_stride, c.page_stride) == (4, 64, 64, 128, 2048)
    turn = lambda t: t.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3)
    _pack4(s=turn, k=turn)
    for kw in (dict(s=turn), dict(k=turn), dict(s=lambda t: t[:, :, :, :1])):
        with pytest.raises(ValueError):
            _pack4(**kw)
    for kw in (dict(s_dt=torch.uint8), dict(k_dt=torch.uint8)):
        with pytest.raises(TypeError):
            _pack4(**kw)
    k = torch.zeros((3, 16, 2, 32), dtype=torch.uint8).view(torch.float4_e2m1fn_x2)
    with pytest.raises(TypeError):
        ds._cache(k.device, k, k)
