"""Pins of the oracle's tree operators and paged cache: closed forms and library routines."""
import numpy as np
import pytest
import torch

from oracle import tree as ot


def _random_parents(rng, T):
    return [-1] + [int(rng.integers(0, i)) for i in range(1, T)]


def test_chain_and_star():
    vis, depth = ot.ancestors([-1, 0, 1, 2])
    assert np.array_equal(vis, np.tril(np.ones((4, 4), bool))) and depth.tolist() == [0, 1, 2, 3]
    vis, depth = ot.ancestors([-1, 0, 0, 0])
    assert np.array_equal(vis, np.eye(4, dtype=bool) | (np.arange(4) == 0)) and depth.tolist() == [0, 1, 1, 1]


@pytest.mark.parametrize("T", [1, 2, 31, 33, 70])
def test_ancestors_are_the_closure_of_the_parent_links(T):
    rng = np.random.default_rng(T)
    parent = _random_parents(rng, T)
    vis, depth = ot.ancestors(parent)
    link = np.eye(T, dtype=np.int64)
    for i in range(1, T):
        link[i, parent[i]] = 1
    closure = np.eye(T, dtype=np.int64)
    for _ in range(T):
        closure = ((closure @ link) > 0).astype(np.int64)
    assert np.array_equal(vis, closure > 0)
    assert np.array_equal(depth, vis.sum(1) - 1)
    words = ot.pack(vis).view(np.uint32)
    assert np.array_equal(((words[:, np.arange(T) // 32] >> (np.arange(T) % 32).astype(np.uint32)) & 1) == 1, vis)


def test_accept_hand_worked():
    #        0
    #      1   2
    #     3 4   5      two children of 1 share a token: the lower index wins
    parent = [-1, 0, 0, 1, 1, 2]
    tok = [9, 11, 12, 13, 13, 15]
    assert ot.accept(parent, tok, [11, 13, 0, 21, 22, 0]) == ([0, 1, 3], [11, 13, 21])
    assert ot.accept(parent, tok, [12, 0, 15, 0, 0, 7]) == ([0, 2, 5], [12, 15, 7])
    assert ot.accept(parent, tok, [99, 0, 0, 0, 0, 0]) == ([0], [99])
    assert ot.accept([], [], []) == ([], [])


def test_attend_is_softmax_attention():
    rng = np.random.default_rng(0)
    q, K, V = rng.standard_normal((3, 4, 8)), rng.standard_normal((5, 2, 8)), rng.standard_normal((5, 2, 8))
    sees = np.array([[1, 1, 0, 1, 1], [0, 0, 1, 0, 0], [0, 0, 0, 0, 0]], bool)
    out, lse, mag, _ = ot.attend(q, K, V, sees, 0.3)
    for h in range(4):
        z = torch.from_numpy(q[:, h] @ K[:, h // 2].T * 0.3).masked_fill(torch.from_numpy(~sees), -np.inf)
        assert np.allclose(lse[:, h], torch.logsumexp(z, 1).numpy())
        assert np.allclose(out[:2, h], torch.softmax(z[:2], 1).numpy() @ V[:, h // 2])
    assert np.allclose(out[1], np.repeat(V[2], 2, 0)) and (out[2] == 0).all() and np.isneginf(lse[2]).all()
    assert (mag >= np.abs(out) - 1e-12).all()


def test_e4m3_matches_torch():
    codes = torch.arange(256, dtype=torch.int32).to(torch.uint8)
    vals = codes.view(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(ot.e4m3_values(), vals, equal_nan=True)
    x = np.concatenate([vals[:127], (vals[:126] + vals[1:127]) / 2, np.linspace(-460, 460, 4001), [0.0, -0.0, 1e-9]])
    x = x.astype(np.float32)
    want = torch.from_numpy(x).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(ot.to_e4m3(x), want)


def test_pool_by_hand():
    c = np.arange(2 * 6 * 4).reshape(2, 6, 4)  # 2 layers, 6 pages of 4 slots
    p = ot.Pool(np.full((3, 3), -1), [0, 0, 0], [0, 0, 0], np.zeros(6, int), 4, [c])
    assert p.reserve([5, 0, 1]) == 1
    assert p.table.tolist() == [[0, 1, -1], [-1, -1, -1], [2, -1, -1]] and p.row_pages.tolist() == [2, 0, 1]
    p.seq_len[:] = [5, 0, 1]
    assert p.fork([-1, 0, -1]) == 1
    assert p.table[1].tolist() == [0, 3, -1] and p.refcount.tolist() == [2, 1, 1, 1, 0, 0] and p.seq_len[1] == 5
    assert np.array_equal(p.caches[0][:, 3, 0], c[:, 1, 0]) and np.array_equal(p.caches[0][:, 3, 1:], c[:, 3, 1:])
    assert p.reserve([0, 0, 12]) == 1 and p.table[2].tolist() == [2, -1, -1]  # row 2 cannot hold 13 of 12
    assert p.reserve([4, 4, 4]) == 0                                          # 3 pages wanted, 2 free
    p.free([1, 0, 1])
    assert p.refcount.tolist() == [1, 0, 0, 1, 0, 0] and p.table[0].tolist() == [-1, -1, -1]
