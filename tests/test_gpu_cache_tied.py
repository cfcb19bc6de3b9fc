"""The cache calls and the attention with one array as both K and V."""
import numpy as np
import pytest
import torch

import draft_selection_amd as ds
from oracle import tree as ot
import test_gpu_cache as tc
import test_gpu_tree_attn as ta

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float8_e4m3fn])
@pytest.mark.parametrize("L,B,T,P,H,D", [(1, 1, 3, 4, 1, 16), (3, 4, 17, 16, 2, 128), (5, 2, 200, 16, 8, 64)])
def test_one_array_as_k_and_v(dev, dt, L, B, T, P, H, D):
    """Appended, compacted and forked once, as a cache of K alone would be."""
    rng = np.random.default_rng(L * T)
    seq = rng.integers(0, 3 * P, B).astype(np.int32)
    cols = int((seq.max() + T + P - 1) // P)
    table = tc._table(rng, B, cols, B * cols + 2)
    k, v = tc._caches(dev, L, B * cols + 2, P, H, D, "tokens", dt)
    new = torch.from_numpy(rng.standard_normal((L, B, T, H, D)).astype(np.float32)).to(dev).to(torch.bfloat16)
    keep = np.stack([np.sort(rng.permutation(T)[:1 + T // 2]) for _ in range(B)])
    path = np.full((B, T), -1, np.int32)
    path[:, :keep.shape[1]] = keep
    d = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(dev)
    n_keep = torch.full((B,), keep.shape[1], dtype=torch.int32, device=dev)
    one = k.clone()
    for a, b in ((k, v), (one, one)):
        ds.cache_append(new, new, a, b, d(table), d(seq))
        ds.cache_compact(a, b, d(table), d(seq), d(path), n_keep)
    assert np.array_equal(tc._bits(one), tc._bits(k))
    for b in range(B):
        for i, j in enumerate(keep[b]):
            p = seq[b] + i
            row = tc._bits(one)[:, table[b, p // P], p % P]
            x = new[:, b, j]
            assert np.array_equal(row, tc._bits(x) if dt == torch.bfloat16 else ot.to_e4m3(x.float().cpu().numpy()))
    t = lambda *a: torch.tensor(a, dtype=torch.int32, device=dev)
    pages = k.shape[1]
    rc = torch.ones(pages, dtype=torch.int32, device=dev)
    rc[-1] = rc[0] = 0
    got = []
    for a, b in ((k, v), (one, one)):
        p = ds.Pages(torch.tensor([[1, -1], [-1, -1]], dtype=torch.int32, device=dev), t(1, 0), t(P - 1, 0), rc.clone(), P)
        assert ds.pages_fork(p, t(-1, 0), a, b).tolist() == [1]
        got.append((tc._bits(a), p.table.tolist(), p.refcount.tolist()))
    assert np.array_equal(got[0][0], got[1][0]) and got[0][1:] == got[1][1:] and ds.device_error() == 0


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float8_e4m3fn])
@pytest.mark.parametrize("ctx", [90, 2000])
def test_attention_over_one_array(dev, dt, ctx):
    rng = np.random.default_rng(ctx)
    q, a, *_ = ta._setup(rng, dev, 2, 9, 8, 2, 128, 16, [ctx, 7], dt)
    a["v_cache"] = a["k_cache"].clone()
    want = ds.tree_attn(q, want_lse=True, **a)
    a["v_cache"] = a["k_cache"]
    got = ds.tree_attn(q, want_lse=True, **a)
    assert all(torch.equal(x, y) for x, y in zip(got, want)) and ds.device_error() == 0
