"""tree_mask and tree_accept on the GPU against the oracle: whole numbers, equal bit for bit."""
import numpy as np
import pytest
import torch

import draft_selection_amd as ds
from oracle import tree as ot

pytestmark = pytest.mark.gpu


def _parents(rng, B, T, kind):
    if kind == "chain":
        p = np.tile(np.arange(-1, T - 1), (B, 1))
    elif kind == "star":
        p = np.zeros((B, T), np.int64)
    else:
        p = np.stack([[-1] + [int(rng.integers(max(0, i - 9), i)) for i in range(1, T)] for _ in range(B)])
    p[:, 0] = -1
    return p.astype(np.int32)


def _case(rng, B, T, kind, vocab=7):
    parent = _parents(rng, B, T, kind)
    tok = rng.integers(0, vocab, (B, T)).astype(np.int32)      # few tokens: siblings share them
    target = rng.integers(0, vocab, (B, T)).astype(np.int32)
    return parent, tok, target


def _ref(parent, tok, target, lens):
    B, T = parent.shape
    n_keep, path, out = np.zeros(B, np.int32), np.full((B, T), -1, np.int32), np.full((B, T), -1, np.int32)
    for b in range(B):
        n = lens[b]
        p, o = ot.accept(parent[b, :n], tok[b, :n], target[b, :n])
        n_keep[b] = len(p)
        path[b, :len(p)], out[b, :len(o)] = p, o
    return n_keep, path, out


@pytest.mark.parametrize("B,T", [(1, 1), (3, 2), (5, 17), (2, 64), (4, 65), (1, 256), (300, 33)])
@pytest.mark.parametrize("kind", ["random", "chain", "star"])
@pytest.mark.parametrize("ragged", [False, True])
def test_mask_and_accept(dev, B, T, kind, ragged):
    rng = np.random.default_rng(B * 1000 + T)
    parent, tok, target = _case(rng, B, T, kind, 2 if kind == "chain" else 7)
    if kind == "chain":
        tok[0] = target[0] = 1                                  # the whole chain is kept
    lens = rng.integers(0, T + 1, B).astype(np.int32) if ragged else np.full(B, T, np.int32)
    d = lambda a: torch.from_numpy(a).to(dev)
    bl = d(lens) if ragged else None
    words = (T + 31) // 32
    mask = torch.full((B, T, words), 77, dtype=torch.int32, device=dev)
    depth = torch.full((B, T), 77, dtype=torch.int32, device=dev)
    ds.tree_mask(d(parent), block_len=bl, out=(mask, depth))
    wide = torch.from_numpy(np.repeat(target[:, :, None], 3, 2).copy()).to(dev)
    wide[:, :, 1:] = -5
    got = ds.tree_accept(d(parent), d(tok), wide[:, :, 0], block_len=bl)
    same = ds.tree_accept(d(parent), d(tok), d(target), block_len=bl)
    torch.cuda.synchronize()
    assert ds.device_error() == 0
    for b in range(B):
        n = lens[b]
        vis, dep = ot.ancestors(parent[b, :n])
        full = np.zeros((n, T), bool)
        full[:, :n] = vis
        words_ref = np.zeros((n, words), np.uint32)
        for j in range(n):
            words_ref[:, j // 32] |= full[:, j].astype(np.uint32) << np.uint32(j % 32)
        assert np.array_equal(mask[b, :n].cpu().numpy(), words_ref.view(np.int32))
        assert np.array_equal(depth[b, :n].cpu().numpy(), dep)
        assert (mask[b, n:] == 77).all() and (depth[b, n:] == 77).all()
    for g, s, r in zip(got, same, _ref(parent, tok, target, lens)):
        assert np.array_equal(g.cpu().numpy(), r) and torch.equal(g, s)


def test_no_tree(dev):
    """Parents that name no earlier node: reported, and their nodes are roots that no path reaches."""
    parent = torch.tensor([[0, 0, 5, -1, 3, -2]], dtype=torch.int32, device=dev)
    tok = torch.zeros((1, 6), dtype=torch.int32, device=dev)
    mask, depth = ds.tree_mask(parent)
    assert ds.device_error() == ds.DEVERR_TREE
    assert mask[0, :, 0].tolist() == [1, 3, 4, 8, 24, 32] and depth[0].tolist() == [0, 1, 0, 0, 1, 0]
    n_keep, path, out = ds.tree_accept(parent, tok, tok)
    assert ds.device_error() == ds.DEVERR_TREE
    assert n_keep.tolist() == [2] and path[0].tolist() == [0, 1, -1, -1, -1, -1] and out[0].tolist() == [0, 0] + [-1] * 4


def test_bad_lengths_make_empty_trees(dev):
    parent = torch.tensor([[-1, 0], [-1, 0], [-1, 0]], dtype=torch.int32, device=dev)
    lens = torch.tensor([3, -1, 2], dtype=torch.int32, device=dev)
    n_keep, path, _ = ds.tree_accept(parent, parent, torch.zeros_like(parent), block_len=lens)
    assert ds.device_error() == ds.DEVERR_BLOCK_LEN
    assert n_keep.tolist() == [0, 0, 2] and path.tolist() == [[-1, -1], [-1, -1], [0, 1]]


def test_empty_batch_and_refusals(dev):
    z = torch.zeros((0, 5), dtype=torch.int32, device=dev)
    assert ds.tree_mask(z)[0].shape == (0, 5, 1) and ds.tree_accept(z, z, z)[0].shape == (0,)
    p = torch.zeros((2, 5), dtype=torch.int32, device=dev)
    with pytest.raises(TypeError):
        ds.tree_mask(p.long())
    with pytest.raises(ds.DselError):
        ds.tree_mask(torch.zeros((1, 257), dtype=torch.int32, device=dev))
    with pytest.raises(ValueError):
        ds.tree_accept(p, p, torch.zeros((2, 10), dtype=torch.int32, device=dev)[:, :5])  # rows not evenly spaced
    with pytest.raises(ValueError):
        ds.tree_mask(p, block_len=torch.zeros(3, dtype=torch.int32, device=dev))


def test_arguments_by_name_and_on_a_stream(dev):
    rng = np.random.default_rng(9)
    parent, tok, target = (torch.from_numpy(x).to(dev) for x in _case(rng, 3, 40, "random"))
    want = ds.tree_mask(parent), ds.tree_accept(parent, tok, target)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = ds.tree_mask(parent=parent, stream=s), ds.tree_accept(target_tok=target, tok=tok, parent=parent, stream=s)
    s.synchronize()
    for x, y in zip(want, got):
        assert all(torch.equal(a, b) for a, b in zip(x, y))
