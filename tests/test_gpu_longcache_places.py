"""The long caches' calls where a cache lies elsewhere: pages past 4 GiB of it, or K and V in turn in one array.  The same
results, bit for bit, as in two small arrays."""
import numpy as np
import pytest
import torch

import draft_selection_amd as ds
import longcache as L

pytestmark = pytest.mark.gpu
P, H, D = 64, 2, 128


def _raw(t):
    return t.view(torch.int16 if t.dtype is L.BF16 else torch.uint8)


@pytest.mark.parametrize("dt", L.TYPES)
def test_pages_past_4_gib(dev, dt):
    rng = np.random.default_rng(1)
    c = L.Case(rng, dev, 3, 6, 8, H, D, P, [700, 64, 333], dt, "tree", room=16)
    N, spare = c.k.shape[0], 24
    moves = dt is L.FP4
    caches = [c.k, c.v] + ([c.k_scale, c.v_scale] if moves else [])
    per = _raw(caches[0])[0].numel() * _raw(caches[0]).element_size()
    far = (5 << 30) // per
    small, big = [], []
    for t in caches:
        for front, out in ((0, small), (far, big)):
            x = torch.empty((front + N + spare, *t.shape[1:]), dtype=_raw(t).dtype, device=dev)
            x[front:front + N] = _raw(t)
            x[front + N:] = 0
            out.append(x.view(t.dtype))
    new = [torch.from_numpy(rng.standard_normal((3, 6, H, D)).astype(np.float32)).to(dev).to(L.BF16) for _ in range(2)]
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device=dev)

    def run(front, t):
        k, v = t[:2]
        ks, vs = t[2:] if moves else (c.k_scale, c.v_scale)
        held = [-(-int(s + n) // P) for s, n in zip(c.seq, c.n)]
        table = torch.full((5, 16), -1, dtype=torch.int32, device=dev)
        for b in range(3):
            table[b, :held[b]] = c.table[b, :held[b]] + front
        got = []
        kw = dict(mask=c.mask, k_scale=ks, v_scale=vs, want_lse=True)
        out, lse = ds.tree_attn(c.q, k, v, table[:3], c.seq_len, **kw)
        got += [out, lse, *ds.tree_attn_window(c.q, k, v, table[:3], c.seq_len, 100, sinks=3, depth=c.depth, **kw)]
        w = torch.zeros((5, 16 * P), device=dev)
        got.append(ds.key_weights(c.q, lse, k, table[:3], c.seq_len, w[:3], k_scale=ks).clone())
        ds.cache_append(*new, k, v, table[:3], c.seq_len, k_scale=ks, v_scale=vs)
        path, keep = i32([[0, 2, 5, -1, -1, -1]] * 3), i32([3, 2, 3])
        lens = ds.cache_compact(k, v, table[:3], c.seq_len, path, keep, k_scale=ks if moves else None, v_scale=vs if moves else None)
        count = torch.zeros(front + N + spare, dtype=torch.int32, device=dev)
        count[:front] = 1
        count[table[table >= 0].long()] = 1
        pages = ds.Pages(table, i32(held + [0, 0]), torch.cat([lens, i32([0, 0])]), count, P)
        mv = dict(k_scale=ks, v_scale=vs) if moves else {}
        got.append(ds.pages_fork(pages, i32([-1, -1, -1, 0, -1]), k, v, **mv))
        got.append(ds.cache_evict(pages, i32([300, -1, 100, 200, -1]), w, k, v, sinks=2, recent=20, **mv))
        got += [torch.where(table >= 0, table - front, table), pages.row_pages, pages.seq_len, count[front:], w]
        got += [_raw(x)[front:].clone() for x in t]
        torch.cuda.synchronize()
        assert ds.device_error() == 0 and (count[:front] == 1).all()
        return got
    a, b = run(0, small), run(far, big)
    for i, (x, y) in enumerate(zip(a, b)):
        x, y = (z.view(torch.int16) if z.dtype is L.BF16 else z for z in (x, y))
        assert torch.equal(x, y), i
    assert a[5].tolist() == [1] and a[6].tolist() == [1]
    c.check(a[0].clone(), a[1].clone())


@pytest.mark.parametrize("dt", L.TYPES)
@pytest.mark.parametrize("between", ["heads", "slots"])
def test_k_and_v_in_turn(dev, dt, between):
    """K and V (and their scale bytes) of a head, or of a slot, side by side."""
    rng = np.random.default_rng(2)
    c = L.Case(rng, dev, 3, 6, 8, H, D, P, [700, 64, 333], dt, "tree", room=16)
    at = -2 if between == "heads" else -3

    def pair(a, b):
        x = torch.stack([_raw(a), _raw(b)], at)
        return x.select(at, 0).view(a.dtype), x.select(at, 1).view(b.dtype)
    scales = (c.k_scale, c.v_scale)
    k, v = pair(c.k, c.v)
    ks, vs = pair(*scales) if dt is L.FP4 else scales
    new = [torch.from_numpy(rng.standard_normal((3, 6, H, D)).astype(np.float32)).to(dev).to(L.BF16) for _ in range(2)]

    def run(k, v, ks, vs):
        kw = dict(mask=c.mask, k_scale=ks, v_scale=vs, want_lse=True)
        out, lse = ds.tree_attn(c.q, k, v, c.table, c.seq_len, **kw)
        got = [out, lse, *ds.tree_attn_window(c.q, k, v, c.table, c.seq_len, 100, sinks=3, depth=c.depth, **kw)]
        w = torch.zeros((3, c.table.shape[1] * P), device=dev)
        got.append(ds.key_weights(c.q, lse, k, c.table, c.seq_len, w, k_scale=ks))
        ds.cache_append(*new, k, v, c.table, c.seq_len, k_scale=ks, v_scale=vs)
        path, keep = (torch.tensor(x, dtype=torch.int32, device=dev) for x in ([[0, 2, 5, -1, -1, -1]] * 3, [3, 2, 3]))
        mv = dict(k_scale=ks, v_scale=vs) if dt is L.FP4 else {}
        got.append(ds.cache_compact(k, v, c.table, c.seq_len, path, keep, **mv))
        torch.cuda.synchronize()
        assert ds.device_error() == 0
        return [x.clone() for x in got] + [_raw(x).clone() for x in ((k, v, ks, vs) if dt is L.FP4 else (k, v))]
    for i, (x, y) in enumerate(zip(run(c.k, c.v, *scales), run(k, v, ks, vs))):
        x, y = (z.view(torch.int16) if z.dtype is L.BF16 else z for z in (x, y))
        assert torch.equal(x, y), i
