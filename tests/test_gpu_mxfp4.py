"""Caches held in 4 bits on the GPU: what appending writes (codes and scales exactly), rows that move with their
scales, and attention over such a cache against the fp64 oracle (bounds: longcache.py)."""
import numpy as np
import pytest
import torch

import draft_selection_amd as ds
import longcache as L
from oracle import longcache as lc

pytestmark = pytest.mark.gpu
E8M0 = torch.float8_e8m0fnu


def _bf16(x, dev):
    return torch.from_numpy(np.asarray(x, np.float32)).to(dev).to(torch.bfloat16)


def _append(dev, x):
    """Codes and scale bytes of bf16 values ``x [n, D]`` (a tensor), appended as one row of n tokens with one head."""
    n, D = x.shape
    k, ks = L.empty_cache(dev, L.FP4, 1, n, 1, D)
    v, vs = L.empty_cache(dev, L.FP4, 1, n, 1, D)
    z = torch.zeros((1, 1), dtype=torch.int32, device=dev)
    new = x.view(1, n, 1, D)
    ds.cache_append(new, new, k, v, z, z[0], k_scale=ks, v_scale=vs)
    torch.cuda.synchronize()
    assert ds.device_error() == 0
    assert torch.equal(k.view(torch.uint8), v.view(torch.uint8)) and torch.equal(ks.view(torch.uint8), vs.view(torch.uint8))
    return lc.unpack(k.view(torch.uint8)[0, :, 0].cpu().numpy()), ks.view(torch.uint8)[0, :, 0].cpu().numpy()


def _same(dev, x):
    x = x.contiguous()
    code, byte = _append(dev, x)
    want_c, want_b = lc.to_mxfp4(x.double().cpu().numpy())
    np.testing.assert_array_equal(byte, want_b)
    # a zero of either sign
    np.testing.assert_array_equal(np.where(code == 8, 0, code), np.where(want_c == 8, 0, want_c))


@pytest.mark.parametrize("e", [-123, -122, -60, 0, 1, 77, 124, 125])
def test_every_value_under_a_scale(dev, e):
    """Every bf16 pattern that fits under 2^e, in blocks whose first value sets that scale."""
    bits = np.arange(1 << 16, dtype=np.uint32) << 16
    v = bits.view(np.float32)
    v = v[np.isfinite(v) & (np.abs(v) <= 7.0 * 2.0 ** e)]
    x = np.full(((len(v) + 30) // 31, 32), 0.0, np.float32)
    flat = np.zeros(x.shape[0] * 31, np.float32)
    flat[:len(v)] = v
    x[:, 1:] = flat.reshape(-1, 31)
    x[:, 0] = 7.0 * 2.0 ** e
    _same(dev, _bf16(x, dev))


def test_scales_of_every_largest_value(dev):
    """Every bf16 pattern as the largest of its block, beside smaller ones of every sign."""
    bits = np.arange(0x7F80, dtype=np.uint32) << 16
    top = bits.view(np.float32)
    rng = np.random.default_rng(0)
    x = top[:, None] * np.concatenate([np.ones((len(top), 1)), rng.uniform(-1, 1, (len(top), 31))], 1).astype(np.float32)
    _same(dev, _bf16(x, dev))


def test_specials_make_their_block_nan(dev):
    x = np.ones((7, 96), np.float32)
    x[0, 3], x[1, 40], x[2, 95], x[3, 64], x[4, :] = np.nan, np.inf, -np.inf, 3.4e38, 0.0
    x[5, 32:64] = -0.0
    _same(dev, _bf16(x, dev))


@pytest.mark.parametrize("layout", ["tokens", "heads", "padded"])
@pytest.mark.parametrize("D,H,P,T", [(32, 1, 8, 3), (96, 3, 5, 9), (128, 8, 16, 70), (256, 2, 64, 130)])
def test_append_places(dev, D, H, P, T, layout):
    """Ragged rows of two layers from strided new rows; what is not written stays."""
    rng = np.random.default_rng(D + T)
    B, layers = 3, 2
    seq, lens = np.array([0, 13, 2 * P], np.int32), np.array([T, 0, max(1, T - 2)], np.int32)
    cols = int(seq.max() + T + P - 1) // P
    table = rng.permutation(B * cols + 2)[:B * cols].reshape(B, cols).astype(np.int32)
    k, ks = L.empty_cache(dev, L.FP4, B * cols + 2, P, H, D, layout, layers)
    v, vs = L.empty_cache(dev, L.FP4, B * cols + 2, P, H, D, layout, layers)
    new = _bf16(rng.standard_normal((layers, B, H, T, 2, D)), dev).transpose(2, 3)   # K and V of a head side by side
    before = [t.view(torch.uint8).cpu().numpy().copy() for t in (k, ks, v, vs)]
    ds.cache_append(new[:, :, :, :, 0], new[:, :, :, :, 1], k, v, L.dev_of(table, dev), L.dev_of(seq, dev),
                    block_len=L.dev_of(lens, dev), k_scale=ks, v_scale=vs)
    torch.cuda.synchronize()
    assert ds.device_error() == 0
    for i, (c, s) in enumerate(((k, ks), (v, vs))):
        want, wantb = before[2 * i].copy(), before[2 * i + 1].copy()
        for b in range(B):
            for t in range(lens[b]):
                pos = seq[b] + t
                code, byte = lc.to_mxfp4(new[:, b, t, :, i].double().cpu().numpy())
                want[:, table[b, pos // P], pos % P], wantb[:, table[b, pos // P], pos % P] = lc.pack(code), byte
        got = c.view(torch.uint8).cpu().numpy()
        code = lc.unpack(got), lc.unpack(want)      # a zero of either sign
        np.testing.assert_array_equal(np.where(code[0] == 8, 0, code[0]), np.where(code[1] == 8, 0, code[1]))
        np.testing.assert_array_equal(s.view(torch.uint8).cpu().numpy(), wantb)


@pytest.mark.parametrize("layout", ["tokens", "heads", "padded"])
def test_compact_moves_scales(dev, layout):
    rng = np.random.default_rng(5)
    layers, pages, P, H, D, T = 3, 9, 4, 2, 96, 11
    k, ks = L.empty_cache(dev, L.FP4, pages, P, H, D, layout, layers)
    v, vs = L.empty_cache(dev, L.FP4, pages, P, H, D, layout, layers)
    for t in (k, ks, v, vs):
        t.view(torch.uint8).copy_(L.dev_of(rng.integers(0, 256, t.shape).astype(np.uint8), dev))
    table = rng.permutation(pages)[:8].reshape(2, 4).astype(np.int32)
    seq = np.array([3, 5], np.int32)
    path, n = np.full((2, T), -1, np.int32), np.array([4, 3], np.int32)
    path[0, :4], path[1, :3] = [0, 3, 4, 10], [2, 3, 9]
    want = [t.view(torch.uint8).cpu().numpy().copy() for t in (k, ks, v, vs)]
    for w in want:
        for b in range(2):
            for i in range(n[b]):
                a, c = seq[b] + path[b, i], seq[b] + i
                w[:, table[b, c // P], c % P] = w[:, table[b, a // P], a % P]
    got = ds.cache_compact(k, v, L.dev_of(table, dev), L.dev_of(seq, dev), L.dev_of(path, dev), L.dev_of(n, dev),
                           k_scale=ks, v_scale=vs)
    assert got.tolist() == [7, 8] and ds.device_error() == 0
    for t, w in zip((k, ks, v, vs), want):
        np.testing.assert_array_equal(t.view(torch.uint8).cpu().numpy(), w)


def test_fork_copies_scales(dev):
    rng = np.random.default_rng(6)
    layers, pages, P, H, D = 2, 8, 24, 3, 64
    caches = [t for _ in range(2) for t in L.empty_cache(dev, L.FP4, pages, P, H, D, "heads", layers)]
    for t in caches:
        t.view(torch.uint8).copy_(L.dev_of(rng.integers(0, 256, t.shape).astype(np.uint8), dev))
    k, ks, v, vs = caches
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device=dev)
    pages_ = ds.Pages(i32([[5, 3, -1], [-1, -1, -1]]), i32([2, 0]), i32([P + 19, 0]), i32([1, 0, 0, 1, 0, 1, 0, 0]), P)
    want = [t.view(torch.uint8).cpu().numpy().copy() for t in caches]
    for w in want:
        w[:, 1, :19] = w[:, 3, :19]
    assert ds.pages_fork(pages_, i32([-1, 0]), k, v, k_scale=ks, v_scale=vs).tolist() == [1]
    assert pages_.table.tolist() == [[5, 3, -1], [5, 1, -1]] and ds.device_error() == 0
    for t, w in zip(caches, want):
        np.testing.assert_array_equal(t.view(torch.uint8).cpu().numpy(), w)


@pytest.mark.parametrize("Hq,H,D", [(1, 1, 128), (4, 1, 128), (10, 2, 128), (8, 8, 64), (16, 2, 256), (3, 3, 96), (5, 1, 32),
                                    (2, 1, 160)])
@pytest.mark.parametrize("layout", ["tokens", "heads", "padded"])
def test_attention_heads(dev, Hq, H, D, layout):
    for room in (0, 4096):
        L.Case(np.random.default_rng(Hq * 1000 + D), dev, 3, 7, Hq, H, D, 16, [0, 93, 300], L.FP4, layout=layout,
               room=room // 16).run()


@pytest.mark.parametrize("T,Hq,H,D", [(1, 4, 1, 64), (1, 32, 8, 128), (9, 4, 1, 64), (17, 8, 2, 128), (16, 8, 1, 128),
                                      (33, 4, 1, 128), (70, 2, 1, 64), (64, 6, 2, 256), (8, 8, 1, 256), (256, 2, 1, 128)])
@pytest.mark.parametrize("kind", ["chain", "tree", "random"])
def test_attention_rows(dev, T, Hq, H, D, kind):
    """Every choice of kernel, rows that see nothing, ragged blocks and an empty one."""
    rng = np.random.default_rng(T * 10 + D)
    L.Case(rng, dev, 4, T, Hq, H, D, 32, [0, 5, 401, 130], L.FP4, kind, lens=[T, max(1, T // 2), T, 0], room=64).run()


@pytest.mark.parametrize("P", [1, 5, 16, 48, 200])
def test_attention_pages(dev, P):
    L.Case(np.random.default_rng(P), dev, 3, 5, 8, 2, 128, P, [255, 64, 511], L.FP4, layout="heads", room=4096 // P).run()


def test_attention_of_long_rows(dev):
    """Rows split over many workgroups, of lengths far apart."""
    c = L.Case(np.random.default_rng(8), dev, 3, 3, 4, 1, 128, 64, [30000, 1, 7000], L.FP4, layout="heads")
    c.run()


def test_attention_beside_many_rows(dev):
    rng = np.random.default_rng(9)
    c = L.Case(rng, dev, 130, 2, 4, 2, 64, 16, rng.integers(0, 200, 130), L.FP4, "chain", lens=rng.integers(0, 3, 130))
    c.run()


def test_unseen_nan_and_infinite_blocks(dev):
    """NaN blocks (scale byte 255) at keys that a node does not see never reach it; at those it sees they do."""
    c = L.Case(np.random.default_rng(3), dev, 1, 6, 4, 2, 128, 16, [37], L.FP4, "random", room=64)
    hidden = 3                                   # no node sees node 3 but those whose bit is set
    c.vis[0, :, hidden] = False
    from oracle import tree as ot
    c.mask = L.dev_of(ot.pack(c.vis), dev)
    rows = c.places(c.table_np, 0, np.array([37 + hidden]))
    c.k_scale.view(torch.uint8)[rows] = 255
    c.v_scale.view(torch.uint8)[rows] = 255
    c.run()
    # now one that node 4 alone sees: its row is NaN, the others are as before
    c.vis[0, 4, hidden] = True
    c.mask = L.dev_of(ot.pack(c.vis), dev)
    want, wl = (t.clone() for t in c.attend())
    c.vis[0, 4, hidden] = False
    c.mask = L.dev_of(ot.pack(c.vis), dev)
    out, lse = c.attend()
    assert torch.isnan(want[0, 4]).all() and torch.isnan(wl[0, 4]).all()
    keep = [0, 1, 2, 3, 5]
    assert torch.equal(want[0, keep], out[0, keep]) and torch.equal(wl[0, keep], lse[0, keep])
    # V alone: one block of 32 columns of the heads that read it
    c.k_scale.view(torch.uint8)[rows] = 127
    c.v_scale.view(torch.uint8)[rows] = 127
    c.v_scale.view(torch.uint8)[(*rows, 1, 2)] = 255
    c.vis[0, 4, hidden] = True
    c.mask = L.dev_of(ot.pack(c.vis), dev)
    out, lse = c.attend()
    bad = torch.isnan(out[0, 4])
    assert bad[2:, 64:96].all() and not bad[:2].any() and not bad[2:, :64].any() and not bad[2:, 96:].any()
    assert torch.isfinite(lse[0, 4]).all() and torch.isfinite(out[0, keep]).all()


def test_bad_pages_are_seen_by_nobody(dev):
    c = L.Case(np.random.default_rng(4), dev, 2, 5, 4, 1, 128, 16, [40, 64], L.FP4, "chain", room=64)
    c.table[0, 1] = -1
    c.table[1, 2] = 1 << 20
    out, lse = c.attend()
    torch.cuda.synchronize()
    assert ds.device_error() == ds.DEVERR_PAGE
    for b, gone in ((0, range(16, 32)), (1, range(32, 48))):
        full = c.sees(b)
        full[:, list(gone)] = False
        c.sees_now = full
        ref = L.ot.attend(c.q[b].double().cpu().numpy(), c.K[b], c.V[b], full, 128 ** -0.5)
        np.testing.assert_allclose(out[b].double().cpu().numpy(), ref[0], atol=0.02, rtol=0.02)
        np.testing.assert_allclose(lse[b].double().cpu().numpy(), ref[1], atol=1e-4)


def test_one_array_as_k_and_v(dev):
    c = L.Case(np.random.default_rng(12), dev, 2, 5, 4, 1, 128, 16, [40, 301], L.FP4, room=64)
    c.v, c.v_scale, c.V = c.k, c.k_scale, c.K
    c.run()


def test_repeats_and_streams(dev):
    c = L.Case(np.random.default_rng(13), dev, 5, 17, 8, 2, 128, 16, [900, 4, 77, 3000, 1200], L.FP4, "chain", layout="heads")
    out, lse = c.attend()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o2, l2 = c.attend(stream=side)
    torch.cuda.synchronize()
    assert torch.equal(out, o2) and torch.equal(lse, l2)


def test_captured_step(dev):
    """Append and attention in one graph, replayed on changed inputs beside eager calls."""
    rng = np.random.default_rng(14)
    c = L.Case(rng, dev, 3, 4, 8, 2, 128, 16, [50, 700, 0], L.FP4, "chain")
    new = [_bf16(rng.standard_normal((3, 4, 2, 128)), dev) for _ in range(2)]
    out, lse = torch.zeros_like(c.q), torch.zeros((3, 4, 8), device=dev)

    def step():
        ds.cache_append(*new, c.k, c.v, c.table, c.seq_len, k_scale=c.k_scale, v_scale=c.v_scale)
        c.attend(out=out, lse=lse)
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for i in range(4):
        for t in new + [c.q]:
            t.copy_(_bf16(rng.standard_normal(t.shape), dev))
        g.replay()
        torch.cuda.synchronize()
        got = out.clone(), lse.clone()
        out.zero_(), lse.zero_()
        step()
        torch.cuda.synchronize()
        assert torch.equal(got[0], out) and torch.equal(got[1], lse), i
