"""key_weights and cache_evict on the GPU against the oracle, and a whole run of the long caches' calls (bounds:
longcache.py)."""
import numpy as np
import pytest
import torch

import draft_selection_amd as ds
import longcache as L
from oracle import longcache as lc

pytestmark = pytest.mark.gpu


def _weigh(c, decay=1.0, count=None, extra=3, seed=0, stream=None):
    rng = np.random.default_rng(seed)
    out, lse = c.attend()
    torch.cuda.synchronize()
    n = c.table.shape[1] * c.P + extra
    before = rng.uniform(0, 2, (c.B, n)).astype(np.float32)
    if decay == 0:
        before[:, 0::3] = np.nan
    w = L.dev_of(before, c.dev)
    if stream is not None:
        stream.wait_stream(torch.cuda.current_stream())
    got = ds.key_weights(c.q, lse, c.k, c.table, c.seq_len, w, block_len=c.block_len, decay=decay, k_scale=c.k_scale,
                         count=None if count is None else L.dev_of(count.astype(np.float32), c.dev), stream=stream)
    torch.cuda.synchronize()
    assert got.data_ptr() == w.data_ptr()
    return w, before.astype(np.float64), lse


def _run(c, decay=1.0, count=None):
    w, before, lse = _weigh(c, decay, count)
    assert ds.device_error() == 0
    L.check_weights(c, w.double().cpu().numpy(), before, lse.double().cpu().numpy(), decay, count)


@pytest.mark.parametrize("dt", L.TYPES)
@pytest.mark.parametrize("T,Hq,H,D", [(1, 1, 1, 128), (1, 32, 8, 128), (9, 10, 2, 128), (17, 8, 8, 64), (8, 8, 1, 256),
                                      (40, 6, 3, 96), (3, 5, 5, 32), (256, 2, 1, 64)])
def test_weights(dev, dt, T, Hq, H, D):
    _run(L.Case(np.random.default_rng(T + D), dev, 4, T, Hq, H, D, 16, [0, 5, 401, 130], dt, lens=[T, max(1, T // 2), T, 0]))


@pytest.mark.parametrize("dt", L.TYPES)
@pytest.mark.parametrize("decay", [0.0, 0.25])
def test_decay_and_counts(dev, dt, decay):
    rng = np.random.default_rng(1)
    count = rng.uniform(0, 2, (3, 6)).astype(np.float32)
    count[0, 2], count[1, :], count[2, 0] = 0, 0, 1e-20
    _run(L.Case(rng, dev, 3, 6, 4, 2, 64, 16, [33, 200, 64], dt, "chain"), decay, count.astype(np.float64))


@pytest.mark.parametrize("layout,P", [("heads", 16), ("padded", 16), ("tokens", 1), ("tokens", 48), ("heads", 200)])
def test_weights_of_layouts_and_pages(dev, layout, P):
    for dt in L.TYPES:
        _run(L.Case(np.random.default_rng(P), dev, 2, 3, 4, 2, 128, P, [300, 77], dt, layout=layout))


def test_weights_of_long_rows(dev):
    for dt in L.TYPES:
        _run(L.Case(np.random.default_rng(2), dev, 2, 2, 4, 1, 64, 64, [20000, 4097], dt))


def test_a_wide_table(dev):
    """Room for far more positions than there are: the rows' work goes round over a bounded grid."""
    _run(L.Case(np.random.default_rng(3), dev, 2, 2, 4, 1, 64, 8, [900, 8000], L.BF16, room=1 << 20))


@pytest.mark.parametrize("dt", L.TYPES)
def test_nodes_that_saw_nothing_or_nan_count_nothing(dev, dt):
    c = L.Case(np.random.default_rng(4), dev, 2, 4, 4, 2, 64, 16, [0, 50], dt, "random")
    c.q[1, 2, 1] = float("nan")
    c.q[1, 3, 0, 5] = float("inf")
    w, before, lse = _weigh(c)
    assert not torch.isfinite(lse[1, 2, 1])
    q = c.q.clone()
    q[1, 2, 1] = 0
    q[1, 3, 0] = 0
    c.q, keep = q, c.q
    got = w.double().cpu().numpy()
    assert np.isfinite(got).all()
    L.check_weights(c, got, before, lse.double().cpu().numpy(), 1.0)


def test_weights_of_bad_pages_and_lengths(dev):
    c = L.Case(np.random.default_rng(5), dev, 3, 2, 4, 2, 64, 16, [50, 40, 20], L.BF16, "chain")
    out, lse = c.attend()
    n = c.table.shape[1] * 16
    w = torch.full((3, n), 2.0, device=dev)
    c.table[0, 1] = -4
    c.seq_len[1] = n + 1
    ds.key_weights(c.q, lse, c.k, c.table, c.seq_len, w)
    torch.cuda.synchronize()
    assert ds.device_error() == ds.DEVERR_PAGE | ds.DEVERR_SEQ_LEN
    assert (w[1] == 2).all() and (w[0, 16:32] == 2).all() and (w[0, 50:] == 2).all()
    assert (w[0, :16] > 2).all() and (w[0, 32:50] > 2).all() and (w[2, :20] > 2).all()


def test_weights_repeat_and_streams(dev):
    c = L.Case(np.random.default_rng(6), dev, 3, 9, 8, 4, 128, 16, [900, 44, 77], L.E4M3, "chain")
    a = _weigh(c)[0]
    b = _weigh(c, stream=torch.cuda.Stream())[0]
    assert torch.equal(a, b)


# ---- eviction ---------------------------------------------------------------------


def _pool(rng, dev, seq, P, cols, spare, layers=2, H=2, D=64, dt=L.BF16, layout="tokens", shared=False):
    """(ds.Pages, k, v, scales, oracle pool): rows of these lengths in a shuffled pool with `spare` free pages."""
    R = len(seq)
    held = [-(-s // P) for s in seq]
    ids = rng.permutation(sum(held) + spare)
    table, ref, at = np.full((R, cols), -1, np.int32), np.zeros(len(ids), np.int32), 0
    for r in range(R):
        table[r, :held[r]] = ids[at:at + held[r]]
        at += held[r]
    if shared:  # row 1 shares its whole pages with row 0
        whole = min(seq[0], seq[1]) // P
        table[1, :whole] = table[0, :whole]
    for r in range(R):
        for p in table[r, :held[r]]:
            ref[p] += 1
    k, ks = L.empty_cache(dev, dt, len(ids), P, H, D, layout, layers)
    v, vs = L.empty_cache(dev, dt, len(ids), P, H, D, layout, layers)
    raw = [t.view(torch.int16 if dt is L.BF16 else torch.uint8) for t in (k, v)] + \
        [t.view(torch.uint8) for t in (ks, vs) if t is not None]
    for t in raw:
        t.copy_(torch.from_numpy(rng.integers(0, 256, t.shape)).to(dev).to(t.dtype))
    seq = np.array(seq, np.int32)
    pool = lc.LongPool(table, np.array(held, np.int32), seq, ref, P, [t.cpu().numpy() for t in raw])
    d = lambda a: L.dev_of(a, dev)
    return ds.Pages(d(table), d(np.array(held, np.int32)), d(seq), d(ref), P), k, v, ks, vs, raw, pool


def _evict(rng, dev, seq, budget, P, cols, spare, sinks, recent, weights=None, extra=2, kept=True, **kw):
    pages, k, v, ks, vs, raw, pool = _pool(rng, dev, seq, P, cols, spare, **kw)
    n = cols * P + extra
    w = np.round(np.exp(2 * rng.standard_normal((len(seq), n))), 1).astype(np.float32) if weights is None else weights.copy()
    wd = L.dev_of(w, dev)
    kd = torch.full((len(seq), n), -5, dtype=torch.int32, device=dev) if kept else None
    got = ds.cache_evict(pages, torch.tensor(budget, dtype=torch.int32, device=dev), wd, k, v, sinks=sinks, recent=recent,
                         k_scale=ks, v_scale=vs, kept=kd)
    torch.cuda.synchronize()
    granted, lists = pool.evict(budget, w, sinks, recent)
    assert got.tolist() == [granted]
    for a, b in ((pages.table, pool.table), (pages.row_pages, pool.row_pages), (pages.seq_len, pool.seq_len),
                 (pages.refcount, pool.refcount), (wd, w)):
        np.testing.assert_array_equal(a.cpu().numpy(), b)
    for t, c in zip(raw, pool.caches):
        np.testing.assert_array_equal(t.cpu().numpy(), c)
    if kept and granted:
        for r, x in enumerate(lists):
            m = 0 if x is None else len(x)
            assert kd[r, :m].tolist() == (x or []) and (kd[r, m:] == -5).all()
    return granted


@pytest.mark.parametrize("dt", L.TYPES)
@pytest.mark.parametrize("layout", ["tokens", "heads", "padded"])
def test_evict(dev, dt, layout):
    rng = np.random.default_rng(0)
    assert _evict(rng, dev, [100, 33, 70, 16, 5], [40, 33, 7, -1, 4], 16, 8, 20, 2, 3, dt=dt, layout=layout) == 1
    assert ds.device_error() == ds.DEVERR_SEQ_LEN    # the last row's 4 cannot hold the 5 that always stay


@pytest.mark.parametrize("P,D,H", [(1, 8, 1), (5, 40, 3), (64, 128, 8), (200, 256, 2)])
def test_evict_geometry(dev, P, D, H):
    rng = np.random.default_rng(P)
    cols = -(-700 // P)
    assert _evict(rng, dev, [700, 257, 64], [400, 256, 1], P, cols, cols * 2, 0, 1, layers=3, D=D, H=H) == 1


@pytest.mark.parametrize("n,keep,sinks,recent", [(5000, 4999, 0, 0), (5000, 1, 0, 0), (5000, 0, 0, 0), (5000, 2500, 2000, 500),
                                                 (1025, 600, 4, 100), (40000, 17000, 1, 0), (1024, 512, 0, 1)])
def test_evict_choices(dev, n, keep, sinks, recent):
    """Long rows, budgets at their edges, ties everywhere, all kinds of weights."""
    rng = np.random.default_rng(n + keep)
    cols = -(-n // 64)
    w = rng.choice(np.array([0, -0.0, 1, 1, 1, 2.5, -3, np.inf, -np.inf, np.nan, -np.nan, 1e-42, 7], np.float32), (2, cols * 64))
    smooth = rng.standard_normal((2, cols * 64)).astype(np.float32)
    for x in (w, smooth, np.zeros_like(w)):
        assert _evict(rng, dev, [n, n - 3], [keep, -1], 64, cols, cols, sinks, recent, weights=x, layers=1, H=1, D=8, extra=0) == 1


def test_evict_shared_pages(dev):
    """A row cut down leaves the pages that another row holds as they are."""
    rng = np.random.default_rng(3)
    assert _evict(rng, dev, [90, 70, 40], [30, -1, -1], 16, 8, 4, 1, 1, shared=True) == 1
    assert _evict(rng, dev, [90, 70, 40], [30, 30, 30], 16, 8, 8, 1, 1, shared=True) == 1


def test_evict_all_or_none(dev):
    rng = np.random.default_rng(4)
    assert _evict(rng, dev, [90, 70], [40, 40], 16, 8, 6, 0, 0) == 1
    assert ds.device_error() == 0
    assert _evict(rng, dev, [90, 70], [40, 40], 16, 8, 5, 0, 0, kept=False) == 0
    assert ds.device_error() == ds.DEVERR_POOL
    assert _evict(rng, dev, [90, 70], [90, 1000], 16, 8, 0, 0, 0) == 1
    assert ds.device_error() == 0


def test_evict_leaves_bad_rows(dev):
    rng = np.random.default_rng(5)
    assert _evict(rng, dev, [90, 70], [40, 4], 16, 8, 9, 3, 2) == 1           # row 1 cannot hold what always stays
    assert ds.device_error() == ds.DEVERR_SEQ_LEN
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device=dev)
    k = torch.zeros((1, 9, 4, 1, 8), device=dev, dtype=torch.bfloat16)
    v = torch.zeros_like(k)
    # a page id that is none; more positions than pages; more pages than the table holds
    pages = ds.Pages(i32([[0, 99, -1], [1, 2, -1], [3, 4, 5]]), i32([2, 2, 4]), i32([7, 9, 9]), i32([1, 1, 1, 1, 1, 1, 0, 0, 0]), 4)
    was = [t.clone() for t in pages[:4]]
    w = torch.ones((3, 12), device=dev)
    assert ds.cache_evict(pages, i32([3, 3, 3]), w, k, v).tolist() == [1]
    assert ds.device_error() == ds.DEVERR_SEQ_LEN | ds.DEVERR_PAGE
    for a, b in zip(pages[:4], was):
        assert torch.equal(a, b)
    assert (w == 1).all()


def test_evict_one_array_as_k_and_v_and_no_rows(dev):
    rng = np.random.default_rng(6)
    pages, k, v, ks, vs, raw, pool = _pool(rng, dev, [50], 16, 4, 4, layers=1)
    w = rng.standard_normal((1, 64)).astype(np.float32)
    assert ds.cache_evict(pages, torch.tensor([20], dtype=torch.int32, device=dev), L.dev_of(w, dev), k, k).tolist() == [1]
    pool.evict([20], w, 0, 0)
    np.testing.assert_array_equal(raw[0].cpu().numpy(), pool.caches[0])
    e = torch.zeros(0, dtype=torch.int32, device=dev)
    none = ds.Pages(torch.zeros((0, 4), dtype=torch.int32, device=dev), e, e, pages.refcount, 16)
    assert ds.cache_evict(none, e, torch.zeros((0, 64), device=dev), k, v).tolist() == [1]


@pytest.mark.parametrize("dt", L.TYPES)
def test_a_whole_run(dev, dt):
    """Drafts appended, attended, weighed and cut down, step after step, in one graph-free loop: what the attention
    gives after the cut is that of a softmax over the kept positions."""
    rng = np.random.default_rng(7)
    B, T, Hq, H, D, P, cols = 2, 3, 4, 2, 64, 16, 8
    layers, budget = 2, 48
    N = B * cols * 2
    k, kb = L.empty_cache(dev, dt, N, P, H, D, "tokens", layers)
    v, vb = L.empty_cache(dev, dt, N, P, H, D, "tokens", layers)
    scale = torch.full((layers, H), 0.02, device=dev) if dt is L.E4M3 else None
    ks, vs = (kb, vb) if dt is L.FP4 else (scale, scale)
    z = lambda *s: torch.zeros(s, dtype=torch.int32, device=dev)
    pages = ds.Pages(torch.full((B, cols), -1, dtype=torch.int32, device=dev), z(B), z(B), z(N), P)
    w = torch.zeros((B, cols * P), device=dev)
    held = [[] for _ in range(B)]                        # what every cached position holds: [layers, 2, H, D]
    sums = np.zeros((B, cols * P))
    wide = lambda a: a[0] if dt is L.BF16 else lc.from_mxfp4(*lc.to_mxfp4(a[0])) if dt is L.FP4 else None
    of = lambda t, i: None if t is None else t[i]
    for step in range(26):
        n = torch.full((B,), T, dtype=torch.int32, device=dev)
        assert ds.pages_reserve(pages, n).tolist() == [1]
        kn, vn = (torch.from_numpy(rng.standard_normal((layers, B, T, H, D)).astype(np.float32)).to(dev).to(L.BF16) for _ in range(2))
        ds.cache_append(kn, vn, k, v, pages.table, pages.seq_len, k_scale=ks, v_scale=vs)
        new = []
        for x in (kn, vn):
            y = x.double().cpu().numpy()
            if dt is L.FP4:
                y = lc.from_mxfp4(*lc.to_mxfp4(y))
            elif dt is L.E4M3:
                y = (x.float() / 0.02).clamp(-448, 448).to(dt).double().cpu().numpy() * float(np.float32(0.02))
            new.append(y)
        for b in range(B):
            held[b] += [np.stack([new[0][:, b, t], new[1][:, b, t]], 1) for t in range(T)]
        for layer in range(layers):
            q = torch.from_numpy(rng.standard_normal((B, T, Hq, D)).astype(np.float32)).to(dev).to(L.BF16)
            out, lse = ds.tree_attn(q, k[layer], v[layer], pages.table, pages.seq_len, k_scale=of(ks, layer),
                                    v_scale=of(vs, layer), want_lse=True)
            ds.key_weights(q, lse, k[layer], pages.table, pages.seq_len, w, k_scale=of(ks, layer), decay=1.0)
            torch.cuda.synchronize()
            for b in range(B):
                have = np.stack(held[b])
                s = len(have) - T
                sees = np.ones((T, s + T), bool)
                sees[:, s:] = np.tril(np.ones((T, T), bool))
                qq = q[b].double().cpu().numpy()
                ref, rl, mag, _ = L.ot.attend(qq, have[:, layer, 0], have[:, layer, 1], sees, D ** -0.5)
                assert np.abs(out[b].double().cpu().numpy() - ref).max() <= 4 * L.HALF * mag.max()
                sums[b, :s] += lc.key_weights(qq, rl, have[:s, layer, 0], D ** -0.5)[0]
        pages.seq_len.add_(T)
        # weights: 26 steps of 2 layers, each within 1e-4 of its sum
        np.testing.assert_allclose(w.double().cpu().numpy(), sums, rtol=2e-4, atol=1e-9)
        if step % 5 == 4:
            kept = torch.full(w.shape, -1, dtype=torch.int32, device=dev)
            m = pages.seq_len.tolist()
            assert ds.cache_evict(pages, torch.full((B,), budget, dtype=torch.int32, device=dev), w, k, v, sinks=1, recent=8,
                                  k_scale=ks, v_scale=vs, kept=kept).tolist() == [1]
            for b in range(B):
                if m[b] > budget:
                    at = kept[b, :budget].tolist()
                    assert at[0] == 0 and at[-8:] == list(range(m[b] - 8, m[b])) and at == sorted(set(at))
                    held[b] = [held[b][i] for i in at]
                    x = sums[b, at]
                    sums[b] = 0
                    sums[b, :budget] = x
                    assert len(held[b]) == int(pages.seq_len[b])
    assert ds.device_error() == 0
    used = int((pages.refcount > 0).sum())
    assert used == int(pages.row_pages.sum()) and used * P <= 2 * B * budget + 6 * P * B


def test_captured_weights_and_eviction(dev):
    """Both in one graph, replayed from the same state beside eager calls."""
    rng = np.random.default_rng(8)
    pages, k, v, ks, vs, raw, pool = _pool(rng, dev, [90, 70, 20], 16, 8, 12, layers=1, dt=L.BF16)
    k.copy_(torch.from_numpy(rng.standard_normal(k.shape).astype(np.float32)).to(dev))
    q = torch.zeros((3, 2, 4, 64), device=dev, dtype=L.BF16)
    w = torch.zeros((3, 128), device=dev)
    budget = torch.tensor([40, 40, 40], dtype=torch.int32, device=dev)
    state = [*pages[:4], w, k, v]
    was = [t.clone() for t in state]

    def step():
        _, lse = ds.tree_attn(q, k[0], v[0], pages.table, pages.seq_len - 2, want_lse=True)
        ds.key_weights(q, lse, k[0], pages.table, pages.seq_len - 2, w)
        return ds.cache_evict(pages, budget, w, k, v, sinks=1, recent=4)

    def back():
        for t, x in zip(state, was):
            t.copy_(x)
        torch.cuda.synchronize()
    step()
    back()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for i in range(4):
        q.copy_(torch.from_numpy(rng.standard_normal(q.shape).astype(np.float32)).to(dev))
        back()
        g.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in state]
        back()
        step()
        torch.cuda.synchronize()
        for a, b in zip(state, got):
            assert torch.equal(a.view(torch.int16) if a.dtype is L.BF16 else a, b.view(torch.int16) if b.dtype is L.BF16 else b), i


def test_evict_many_rows(dev):
    """More rows than the pool's workgroup has threads."""
    rng = np.random.default_rng(30)
    seq = [int(x) for x in rng.integers(0, 13, 1300)]
    budget = [int(x) for x in rng.integers(-1, 9, 1300)]
    assert _evict(rng, dev, seq, budget, 4, 3, 1500, 0, 0, layers=1, H=1, D=8) == 1
    assert ds.device_error() == 0


def test_weights_of_many_rows(dev):
    rng = np.random.default_rng(31)
    _run(L.Case(rng, dev, 130, 2, 4, 2, 64, 16, rng.integers(0, 90, 130), L.FP4, "chain", lens=rng.integers(0, 3, 130)), 0.5)
