"""Pins of the long caches' oracle: worked values, the 4-bit grid, windows, weights and what eviction keeps."""
import numpy as np
import pytest

from oracle import longcache as lc
from oracle import tree as ot


def test_four_bit_codes_by_hand():
    x = np.zeros(64)
    x[:8] = [7, -6, 5, 3.5, 2.5, 1.75, 0.25, -0.26]       # e = 0: 7 is held to 6; ties go to the even code
    x[32:35] = [7.01, 1.0, -0.5]                          # past 7: the next power of two
    code, byte = lc.to_mxfp4(x)
    assert byte.tolist() == [127, 128]
    assert lc.from_mxfp4(code, byte)[:8].tolist() == [6, -6, 4, 4, 2, 2, 0, -0.5]
    assert lc.from_mxfp4(code, byte)[32:35].tolist() == [8, 1, -0.0]   # 7.01 / 2 = 3.505 -> 4; 0.25 ties to 0
    assert lc.unpack(lc.pack(code)).tolist() == code.tolist()


def test_four_bit_grid_is_its_own_image():
    code = np.arange(16, dtype=np.uint8).repeat(2)
    for byte in (4, 100, 127, 200, 252):
        v = lc.from_mxfp4(code, np.array([byte], np.uint8))
        c2, b2 = lc.to_mxfp4(v)
        assert b2.tolist() == [byte] and c2.tolist() == code.tolist()


def test_four_bit_edges():
    zero, small, large = np.zeros(32), np.full(32, 2.0 ** -130), np.full(32, 3.3e38)
    c, b = lc.to_mxfp4(np.concatenate([zero, small, large]))
    assert b.tolist() == [4, 4, 252] and (c[:64] == 0).all() and (c[64:] == 7).all()
    for bad in (np.nan, np.inf, -np.inf):
        x = np.ones(32)
        x[5] = bad
        c, b = lc.to_mxfp4(x)
        assert b.tolist() == [255] and (c == 0).all() and np.isnan(lc.from_mxfp4(c, b)).all()


def test_window_by_hand():
    sees = np.tril(np.ones((3, 3), bool))
    sees = np.concatenate([np.ones((3, 5), bool), sees], 1)           # 5 cached, a chain of 3
    got = lc.window_sees(sees, 5, [0, 1, 2], 3, 1)
    assert got.astype(int).tolist() == [[1, 0, 0, 1, 1, 1, 0, 0], [1, 0, 0, 0, 1, 1, 1, 0], [1, 0, 0, 0, 0, 1, 1, 1]]
    got = lc.window_sees(np.ones((3, 8), bool), 5, [0, 1, 1], 2, 0)   # siblings are at the same position
    assert got.astype(int).tolist() == [[0, 0, 0, 0, 1, 1, 1, 1], [0, 0, 0, 0, 0, 1, 1, 1], [0, 0, 0, 0, 0, 1, 1, 1]]


def test_key_weights_sum_to_the_queries():
    """Over every key that a softmax sees its weights sum to one for each query and head."""
    rng = np.random.default_rng(0)
    q, K = rng.standard_normal((3, 4, 8)), rng.standard_normal((11, 2, 8))
    _, lse, _, _ = ot.attend(q, K, K, np.ones((3, 11), bool), 0.3)
    w, _ = lc.key_weights(q, lse, K, 0.3)
    assert abs(w.sum() - 12) < 1e-12
    w, _ = lc.key_weights(q, lse, K, 0.3, [1.0, 0.0, 0.5])
    assert abs(w.sum() - 6) < 1e-12
    lse[1, 2] = -np.inf
    w, _ = lc.key_weights(q, lse, K, 0.3)
    assert abs(w.sum() - 11) < 1e-12


@pytest.mark.parametrize("w,n,budget,sinks,recent,want", [
    ([1, 5, 2, 5, 0, 3], 6, 3, 0, 0, [1, 3, 5]), ([1, 1, 1, 1, 1, 1], 6, 3, 0, 0, [0, 1, 2]),
    ([9, 1, 2, 3, 9, 0], 6, 4, 1, 2, [0, 3, 4, 5]), ([np.nan, -np.inf, np.nan, 0, 7, 7], 4, 2, 0, 0, [1, 3]),
    ([np.nan, np.nan, -1, 3], 4, 3, 0, 0, [0, 2, 3]), ([3, 2, 1], 3, 0, 0, 0, [])])
def test_kept_positions(w, n, budget, sinks, recent, want):
    assert lc.keep(np.array(w, float), n, budget, sinks, recent) == want


def test_evicted_rows_move_in_order():
    cache = np.arange(2 * 8 * 2).reshape(2, 8, 2)                     # two layers, 8 pages of 2 slots
    pool = lc.LongPool([[5, 1, 3, -1], [5, 2, -1, -1]], [3, 2], [5, 3], [0, 1, 1, 1, 0, 2, 0, 1], 2, [cache])
    w = np.array([[4, 0, 3, 2, 1, 0, 0, 0], [1, 2, 3, 0, 0, 0, 0, 0]], float)
    granted, kept = pool.evict([3, -1], w, 1, 1)
    assert granted == 1 and kept == [[0, 2, 4], None]
    assert pool.table.tolist() == [[0, 4, -1, -1], [5, 2, -1, -1]] and pool.seq_len.tolist() == [3, 3]
    assert pool.refcount.tolist() == [1, 0, 1, 0, 1, 1, 0, 1]
    assert pool.caches[0][0, 0].tolist() == [10, 2] and pool.caches[0][0, 4, 0] == 6
    assert w[0].tolist() == [4, 3, 1, 0, 0, 0, 0, 0]
    assert pool.evict([2, 2], w, 1, 2)[1] == [None, None]             # a budget that cannot hold what always stays
