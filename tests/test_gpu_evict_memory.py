"""cache_evict on arrays that lie in the gaps of each other's rows."""
import numpy as np
import pytest
import torch

import draft_selection_amd as ds
import longcache as L
import test_gpu_evict as te

pytestmark = pytest.mark.gpu


def test_rows_between_rows(dev):
    """Weights, kept positions, budgets and the pool's lengths as columns of one allocation: the same results as apart."""
    rng = np.random.default_rng(0)
    seq, budget, P, cols = [100, 90, 70], [40, -1, 65], 16, 8
    n = cols * P
    w = rng.standard_normal((3, n)).astype(np.float32)
    pages, k, v, ks, vs, raw, pool = te._pool(rng, dev, seq, P, cols, 9)
    slab = torch.full((3, 2 * n + 8), -7, dtype=torch.int32, device=dev)
    wd, kept = slab[:, :n].view(torch.float32), slab[:, n:2 * n]
    wd.copy_(L.dev_of(w, dev))
    gap = slab[1, 2 * n:2 * n + 6]
    gap[:3], gap[3:] = torch.tensor(budget, dtype=torch.int32), pages.seq_len
    pages = pages._replace(seq_len=gap[3:])
    got = ds.cache_evict(pages, gap[:3], wd, k, v, sinks=2, recent=3, kept=kept)
    torch.cuda.synchronize()
    granted, lists = pool.evict(budget, w, 2, 3)
    assert got.tolist() == [granted] == [1] and ds.device_error() == 0
    for a, b in ((pages.table, pool.table), (pages.row_pages, pool.row_pages), (pages.seq_len, pool.seq_len),
                 (pages.refcount, pool.refcount), (wd, w)):
        np.testing.assert_array_equal(a.cpu().numpy(), b)
    for t, c in zip(raw, pool.caches):
        np.testing.assert_array_equal(t.cpu().numpy(), c)
    for r, x in enumerate(lists):
        m = 0 if x is None else len(x)
        assert kept[r, :m].tolist() == (x or []) and (kept[r, m:] == -7).all()
    assert (slab[0, 2 * n:] == -7).all() and (slab[2, 2 * n:] == -7).all() and (slab[1, -2:] == -7).all()
