"""cache_append, cache_compact and the page pool on the GPU against the oracle.

Rows are copies of bits and pages whole numbers, so everything is compared bit
for bit; 8-bit values are the oracle's nearest codes of the fp32 quotient."""
import numpy as np
import pytest
import torch

import draft_selection_amd as ds
from oracle import tree as ot

pytestmark = pytest.mark.gpu


def _caches(dev, layers, pages, P, H, D, layout, dt):
    """K and V of the layout, filled with a pattern; returns views [layers, pages, P, H, D]."""
    it = torch.int16 if dt == torch.bfloat16 else torch.uint8
    n = layers * pages * P * H * D
    pat = (torch.arange(2 * n, device=dev) % 113).to(it)
    if layout == "interleaved":
        x = pat.view(layers, pages, 2, P, H, D)
        k, v = x[:, :, 0], x[:, :, 1]
    else:
        shape = (layers, pages, P, H, D) if layout == "tokens" else (layers, pages, H, P, D)
        k, v = pat[:n].clone().view(shape), pat[n:].clone().view(shape)
        if layout == "heads":
            k, v = k.transpose(2, 3), v.transpose(2, 3)
    return k.view(dt), v.view(dt)


def _bits(x):
    return (x.view(torch.int16) if x.dtype == torch.bfloat16 else x.view(torch.uint8)).cpu().numpy().copy()


def _table(rng, B, cols, pages):
    return rng.permutation(pages)[:B * cols].reshape(B, cols).astype(np.int32)


@pytest.mark.parametrize("layers,B,T,P,H,D", [(1, 1, 1, 16, 1, 8), (1, 3, 5, 7, 2, 40), (2, 4, 17, 16, 8, 128),
                                              (3, 2, 70, 64, 1, 256), (1, 2, 200, 1, 3, 16)])
@pytest.mark.parametrize("layout", ["tokens", "heads", "interleaved"])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float8_e4m3fn])
def test_append_and_compact(dev, layers, B, T, P, H, D, layout, dt):
    if dt == torch.float8_e4m3fn and D % 16:
        D = 16
    rng = np.random.default_rng(T * 10 + B)
    seq = rng.integers(0, 3 * P, B).astype(np.int32)
    cols = int((seq.max() + T + P - 1) // P)
    pages = B * cols + 2
    table = _table(rng, B, cols, pages)
    lens = rng.integers(0, T + 1, B).astype(np.int32)
    lens[-1] = T
    k, v = _caches(dev, layers, pages, P, H, D, layout, dt)
    want = [_bits(k), _bits(v)]
    wide = torch.from_numpy(rng.standard_normal((layers, B, T, 2, H, D)).astype(np.float32)).to(dev)
    wide = wide * torch.from_numpy(np.exp(rng.uniform(-6, 7, (layers, B, T, 2, 1, 1)))).float().to(dev)
    new = wide.to(torch.bfloat16)
    kn, vn = new[:, :, :, 0], new[:, :, :, 1]
    scale = {}
    if dt == torch.float8_e4m3fn:
        scale = {n: torch.from_numpy(rng.uniform(0.3, 3, (layers, H)).astype(np.float32)).to(dev)
                 for n in ("k_scale", "v_scale")}
    d = lambda a: torch.from_numpy(a).to(dev)
    tab, sl = d(table), d(seq)
    one = layers == 1
    cut = (lambda x: x[0]) if one else (lambda x: x)
    ds.cache_append(cut(kn), cut(vn), cut(k), cut(v), tab, sl, block_len=d(lens), **{n: cut(s) for n, s in scale.items()})
    for i, (x, n) in enumerate(((kn, "k_scale"), (vn, "v_scale"))):
        if scale:
            bits = ot.to_e4m3((x.float() / scale[n][:, None, None, :, None]).cpu().numpy())
        else:
            bits = _bits(x.contiguous())
        for b in range(B):
            for t in range(lens[b]):
                p = seq[b] + t
                want[i][:, table[b, p // P], p % P] = bits[:, b, t]
    assert np.array_equal(_bits(k), want[0]) and np.array_equal(_bits(v), want[1])
    # keep an ascending part of each row's tokens
    path, n_keep = np.full((B, T), -1, np.int32), np.zeros(B, np.int32)
    for b in range(B):
        keep = np.sort(rng.permutation(lens[b])[:rng.integers(0, lens[b] + 1)])
        n_keep[b] = len(keep)
        path[b, :len(keep)] = keep
    n_keep[0] = lens[0]
    path[0, :lens[0]] = np.arange(lens[0])
    if T <= ds.MAX_TREE:
        new_len = ds.cache_compact(cut(k), cut(v), tab, sl, d(path), d(n_keep))
        for w in want:
            for b in range(B):
                rows = [w[:, table[b, (seq[b] + j) // P], (seq[b] + j) % P].copy() for j in path[b, :n_keep[b]]]
                for i, r in enumerate(rows):
                    w[:, table[b, (seq[b] + i) // P], (seq[b] + i) % P] = r
        assert np.array_equal(new_len.cpu().numpy(), seq + n_keep)
        assert np.array_equal(_bits(k), want[0]) and np.array_equal(_bits(v), want[1])
    assert ds.device_error() == 0


def test_append_nan_and_range(dev):
    """NaN stays NaN, infinities and large values are held to 448."""
    k = torch.zeros((1, 4, 1, 16), device=dev).to(torch.float8_e4m3fn)
    v = k.clone()
    x = torch.tensor([float("nan"), float("inf"), -float("inf"), 1e30, -449.0, 448.0, 464.0, 2.0 ** -9, 2.0 ** -10,
                      1.5 * 2.0 ** -9, -0.0, 17.0, 18.0, 19.0, 3e38, 1.0], device=dev).to(torch.bfloat16).view(1, 1, 1, 16)
    z = torch.zeros((1, 1), dtype=torch.int32, device=dev)
    ds.cache_append(x, x, k, v, z, z[0])
    got = k[0, 0, 0].float().cpu().numpy()
    want = ot.e4m3_values()[ot.to_e4m3(x.float().cpu().numpy().reshape(-1))]
    assert np.array_equal(got, want, equal_nan=True) and np.isnan(got[0]) and got[1] == 448


def test_rows_that_do_not_fit_are_left(dev):
    k = torch.ones((4, 4, 1, 8), device=dev, dtype=torch.bfloat16)
    v = k.clone()
    x = torch.full((5, 2, 1, 8), 3.0, device=dev, dtype=torch.bfloat16)
    tab = torch.tensor([[0], [1], [9], [-1], [2]], dtype=torch.int32, device=dev)  # one page of 4 slots each
    seq = torch.tensor([3, -1, 0, 0, 2], dtype=torch.int32, device=dev)           # row 0 would pass its page
    ds.cache_append(x, x, k, v, tab, seq)
    assert ds.device_error() == ds.DEVERR_SEQ_LEN | ds.DEVERR_PAGE
    assert (k[[0, 1, 3]] == 1).all() and (k[2, :2] == 1).all() and (k[2, 2:] == 3).all()
    path = torch.tensor([[0, 1], [0, 1], [1, 1], [1, -1], [1, -1]], dtype=torch.int32, device=dev)
    n = torch.tensor([2, 1, 2, 1, 1], dtype=torch.int32, device=dev)
    k[2, 3] = 7
    before = k.clone()
    new = ds.cache_compact(k, v, tab, seq, path, n)
    assert ds.device_error() == ds.DEVERR_SEQ_LEN | ds.DEVERR_PAGE | ds.DEVERR_TREE
    assert new.tolist() == [3, -1, 0, 0, 3]
    before[2, 2] = 7
    assert torch.equal(k, before)
    for bad in (3, -1):
        assert ds.cache_compact(k, v, tab, seq, path, torch.full_like(n, bad)).tolist() == seq.tolist()
        assert ds.device_error() == ds.DEVERR_TREE
    assert torch.equal(k, before)


def test_binding_refusals(dev):
    k = torch.zeros((4, 4, 2, 8), device=dev, dtype=torch.bfloat16)
    x = torch.zeros((1, 2, 2, 8), device=dev, dtype=torch.bfloat16)
    tab, seq = torch.zeros((1, 2), dtype=torch.int32, device=dev), torch.zeros(1, dtype=torch.int32, device=dev)
    ok = dict(k_new=x, v_new=x, k_cache=k, v_cache=k.clone(), page_table=tab, seq_len=seq)
    for kw in (dict(v_cache=k.transpose(1, 2)), dict(v_cache=k[:2]), dict(k_cache=k.float()), dict(k_new=x.float()),
               dict(v_new=x[:, :1]), dict(k_new=x[..., :4], v_new=x[..., :4]), dict(page_table=tab.long()),
               dict(page_table=tab.expand(3, 2)), dict(seq_len=seq.repeat(2)), dict(k_scale=torch.ones(2, device=dev)),
               dict(k_new=x[None], v_new=x[None]), dict(seq_len=seq.cpu())):
        a = {**ok, **kw}
        with pytest.raises((TypeError, ValueError, ds.DselError)):
            ds.cache_append(a.pop("k_new"), **a)


# ------------------------------------------------------------------- pages ---
def _pool(rng, dev, rows, cols, P, spare, layers=2, H=2, D=8, shared=True):
    """A pool in use: rows of all lengths, some pages shared between rows, free ones in between."""
    seq = rng.integers(0, cols * P + 1, rows).astype(np.int32)
    seq[rng.random(rows) < 0.3] = 0
    held = -(-seq // P)
    held = np.minimum(cols, held + rng.integers(0, 2, rows)).astype(np.int32)
    held[seq == 0] = 0
    pages = int(held.sum()) + spare
    ids = rng.permutation(pages)
    table, ref, at = np.full((rows, cols), -1, np.int32), np.zeros(pages, np.int32), 0
    for r in range(rows):
        table[r, :held[r]] = ids[at:at + held[r]]
        at += held[r]
        if shared and r and held[r] and held[r - 1] and seq[r] >= P and seq[r - 1] >= P:
            table[r, 0] = table[r - 1, 0]
        ref[table[r, :held[r]]] += 1
    k = torch.from_numpy(rng.standard_normal((layers, pages, P, H, D)).astype(np.float32)).to(dev).to(torch.bfloat16)
    v = torch.from_numpy(rng.standard_normal((layers, pages, P, H, D)).astype(np.float32)).to(dev).to(torch.bfloat16)
    d = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(dev)
    return (ds.Pages(d(table), d(held), d(seq), d(ref), P), k, v,
            ot.Pool(table, held, seq, ref, P, [_bits(k), _bits(v)]))


def _same(pages, k, v, ref):
    assert np.array_equal(pages.table.cpu().numpy(), ref.table)
    assert np.array_equal(pages.row_pages.cpu().numpy(), ref.row_pages)
    assert np.array_equal(pages.seq_len.cpu().numpy(), ref.seq_len)
    assert np.array_equal(pages.refcount.cpu().numpy(), ref.refcount)
    assert np.array_equal(_bits(k), ref.caches[0]) and np.array_equal(_bits(v), ref.caches[1])


@pytest.mark.parametrize("rows,cols,P,spare", [(1, 1, 16, 3), (2, 3, 1, 9), (7, 5, 16, 40), (40, 9, 7, 30),
                                               (100, 4, 64, 260), (1030, 3, 4, 4000), (4096, 2, 2, 20000)])
def test_pool(dev, rows, cols, P, spare):
    rng = np.random.default_rng(rows + cols)
    pages, k, v, ref = _pool(rng, dev, rows, cols, P, spare)
    d = lambda a: torch.from_numpy(np.asarray(a, np.int32)).to(dev)
    for step in range(4):
        which = (rng.random(rows) < 0.3).astype(np.int32) * rng.integers(1, 9, rows).astype(np.int32)
        ds.pages_free(pages, d(which))
        ref.free(which)
        _same(pages, k, v, ref)
        empty = np.nonzero(ref.row_pages == 0)[0]
        have = np.nonzero(ref.row_pages > 0)[0]
        src = np.full(rows, -1, np.int32)
        if len(empty) and len(have):
            dst = empty[rng.random(len(empty)) < 0.7]
            src[dst] = rng.choice(have, len(dst))
        got = ds.pages_fork(pages, d(src), k, v)
        assert got.tolist() == [ref.fork(src)]
        _same(pages, k, v, ref)
        extra = rng.integers(0, 2 * P, rows)
        extra = np.where(ref.seq_len + extra > cols * P, 0, extra)
        got = ds.pages_reserve(pages, d(extra))
        assert got.tolist() == [ref.reserve(extra)]
        _same(pages, k, v, ref)
        assert ds.device_error() in (0, ds.DEVERR_POOL)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float8_e4m3fn])
@pytest.mark.parametrize("layout", ["heads", "interleaved"])
@pytest.mark.parametrize("P,part", [(16, 15), (16, 1), (40, 33), (64, 64)])
def test_fork_copies_only_what_is_used(dev, dt, layout, P, part):
    """The slots in use of the partial page, every layer and head of any layout; all else stays as it was."""
    k, v = _caches(dev, 3, 6, P, 2, 32, layout, dt)
    want = [_bits(k), _bits(v)]
    t = lambda *a: torch.tensor(a, dtype=torch.int32, device=dev)
    n = 2 * P + part
    p = ds.Pages(torch.tensor([[-1] * 4, [4, 1, 3, -1]], dtype=torch.int32, device=dev), t(0, 3), t(0, n),
                 t(0, 1, 0, 1, 1, 0), P)
    assert ds.pages_fork(p, t(1, -1), k, v).tolist() == [1] and ds.device_error() == 0
    if part < P:
        for w in want:
            w[:, 0, :part] = w[:, 3, :part]
    assert p.table.tolist() == [[4, 1, 0 if part < P else 3, -1], [4, 1, 3, -1]]
    assert p.refcount.tolist() == ([1, 2, 0, 1, 2, 0] if part < P else [0, 2, 0, 2, 2, 0]) and p.seq_len.tolist() == [n, n]
    assert np.array_equal(_bits(k), want[0]) and np.array_equal(_bits(v), want[1])


def test_pool_runs_short(dev):
    """Too few free pages for all rows: nothing changes, and it is said."""
    P = 4
    z = lambda *s: torch.zeros(s, dtype=torch.int32, device=dev)
    pages = ds.Pages(z(3, 4) - 1, z(3), z(3), z(6), P)
    k = torch.zeros((1, 6, P, 1, 8), device=dev, dtype=torch.bfloat16)
    assert ds.pages_reserve(pages, z(3) + 9).tolist() == [0] and ds.device_error() == ds.DEVERR_POOL
    assert (pages.table == -1).all() and (pages.refcount == 0).all() and (pages.row_pages == 0).all()
    assert ds.pages_reserve(pages, torch.tensor([16, 8, 0], dtype=torch.int32, device=dev)).tolist() == [1]
    assert ds.device_error() == 0 and pages.table[0].tolist() == [0, 1, 2, 3] and pages.table[1].tolist() == [4, 5, -1, -1]
    pages.seq_len.copy_(torch.tensor([15, 8, 0], dtype=torch.int32))
    src = torch.tensor([-1, -1, 0], dtype=torch.int32, device=dev)
    assert ds.pages_fork(pages, src, k, k.clone()).tolist() == [0] and ds.device_error() == ds.DEVERR_POOL
    assert pages.row_pages[2] == 0 and (pages.refcount == 1).all()
    src[2] = 1                                           # whole pages only: none is needed
    assert ds.pages_fork(pages, src, k, k.clone()).tolist() == [1] and ds.device_error() == 0
    assert pages.table[2].tolist() == [4, 5, -1, -1] and pages.refcount.tolist() == [1, 1, 1, 1, 2, 2]


def test_bad_entries_are_left_out(dev):
    P = 4
    t = lambda *a: torch.tensor(a, dtype=torch.int32, device=dev)
    k = torch.zeros((1, 9, P, 1, 8), device=dev, dtype=torch.bfloat16)

    def pool():
        return ds.Pages(torch.tensor([[0, 1], [-1, -1], [2, -1], [-1, -1]], dtype=torch.int32, device=dev),
                        t(2, 0, 1, 0), t(8, 0, 4, 0), t(1, 1, 1, 0, 0, 0, 0, 0, 0), P)

    p = pool()
    # row 0 holds pages, row 1's source is itself a target, row 3 names no row
    assert ds.pages_fork(p, t(2, 0, -1, 7), k, k.clone()).tolist() == [1]
    assert ds.device_error() == ds.DEVERR_SEQ_LEN
    assert p.row_pages.tolist() == [2, 0, 1, 0] and p.refcount.tolist() == [1, 1, 1] + [0] * 6
    assert ds.pages_fork(p, t(-1, 1, -1, -3), k, k.clone()).tolist() == [1]
    assert ds.device_error() == ds.DEVERR_SEQ_LEN and p.row_pages.tolist() == [2, 0, 1, 0]
    assert ds.pages_reserve(p, t(1, 4, 4, -1)).tolist() == [1]      # row 0 is full, row 3's wish is no length
    assert ds.device_error() == ds.DEVERR_SEQ_LEN
    assert p.table.tolist() == [[0, 1], [3, -1], [2, 4], [-1, -1]] and p.refcount.tolist() == [1, 1, 1, 1, 1, 0, 0, 0, 0]
    p = pool()
    p.table[2, 0] = 9                                               # no page
    p.refcount[1] = 0                                               # freed once too often
    ds.pages_free(p, t(1, 0, 1, 1))
    assert ds.device_error() == ds.DEVERR_PAGE
    assert (p.refcount == t(0, 0, 1, 0, 0, 0, 0, 0, 0)).all() and (p.table == -1).all() and (p.row_pages == 0).all()
    p = pool()
    p.row_pages[0] = 3
    ds.pages_free(p, t(1, 0, 0, 0))
    assert ds.device_error() == ds.DEVERR_SEQ_LEN and p.refcount.tolist() == [1, 1, 1] + [0] * 6


def test_large_pools(dev):
    """More pages than one pass looks at (16,384), the free ones at the far end."""
    n = 70001
    for left in (5, 40000):
        ref = torch.ones(n, dtype=torch.int32, device=dev)
        ref[n - left:] = 0
        t = torch.full((3, 30000), -1, dtype=torch.int32, device=dev)
        z = torch.zeros(3, dtype=torch.int32, device=dev)
        p = ds.Pages(t, z.clone(), z.clone(), ref, 2)
        want = torch.tensor([3, 0, 2 * left - 5], dtype=torch.int32, device=dev)
        granted = ds.pages_reserve(p, want)
        if left == 5:
            assert granted.tolist() == [1] and t[0, :3].tolist() == [n - 5, n - 4, -1] and t[2, :4].tolist() == [n - 3, n - 2, n - 1, -1]
            assert (ref == 1).all()
        else:
            assert granted.tolist() == [1]      # row 2 cannot hold so many: left out
            assert ds.device_error() == ds.DEVERR_SEQ_LEN and t[0, :2].tolist() == [n - left, n - left + 1]
            want = torch.tensor([3, 50000, 20000], dtype=torch.int32, device=dev)
            assert ds.pages_reserve(p, want).tolist() == [1]
            got = torch.cat([t[1, :25000], t[2, :10000]])
            assert torch.equal(got, torch.arange(n - left + 2, n - left + 2 + 35000, dtype=torch.int32, device=dev))
        assert ds.device_error() == 0
    # wishes whose sum passes 32 bits: none is granted, nothing changes
    rows, cols = 4000, 1 << 20
    t = torch.full((1, cols), -1, dtype=torch.int32, device=dev).expand(rows, cols)
    with pytest.raises(ValueError):
        ds.pages_reserve(ds.Pages(t, ref[:1], ref[:1], ref, 1), ref[:1])  # a table of one shared row is none
    t = torch.full((8, 1 << 29), -1, dtype=torch.int32, device=dev)
    z = torch.zeros(8, dtype=torch.int32, device=dev)
    p = ds.Pages(t, z.clone(), z.clone(), torch.zeros(100, dtype=torch.int32, device=dev), 1)
    assert ds.pages_reserve(p, z + (1 << 29)).tolist() == [0] and ds.device_error() == ds.DEVERR_POOL
    assert (p.row_pages == 0).all() and (p.refcount == 0).all() and (t[:, :4] == -1).all()
    # the same of a pool of more than 2^20 pages, and a wish that it just holds
    ref = torch.zeros((1 << 20) + 5, dtype=torch.int32, device=dev)
    p = ds.Pages(t, z.clone(), z.clone(), ref, 1)
    assert ds.pages_reserve(p, z + (1 << 29)).tolist() == [0] and ds.device_error() == ds.DEVERR_POOL
    want = z.clone()
    want[3], want[5] = 1 << 20, 6
    assert ds.pages_reserve(p, want).tolist() == [0] and ds.device_error() == ds.DEVERR_POOL and (ref == 0).all()
    want[5] = 5
    assert ds.pages_reserve(p, want).tolist() == [1] and ds.device_error() == 0 and (ref == 1).all()
    assert t[5, :6].tolist() == [(1 << 20) + i for i in range(5)] + [-1] and t[3, [0, -1]].tolist() == [0, -1]
    assert p.row_pages.tolist() == [0, 0, 0, 1 << 20, 0, 5, 0, 0]
    del t, p
    e = torch.zeros(0, dtype=torch.int32, device=dev)
    p = ds.Pages(torch.zeros((0, 2), dtype=torch.int32, device=dev), e, e, ref, 2)
    assert ds.pages_reserve(p, e).tolist() == [1]
    ds.pages_free(p, e)
