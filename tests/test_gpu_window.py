"""tree_attn_window on the GPU against the fp64 oracle, in every cache type (bounds: longcache.py)."""
import numpy as np
import pytest
import torch

import draft_selection_amd as ds
import longcache as L

pytestmark = pytest.mark.gpu
BIG = 1 << 62


@pytest.mark.parametrize("dt", L.TYPES)
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (2, 3), (7, 0), (40, 4), (128, 0), (300, 70), (BIG, 0), (5, BIG)])
@pytest.mark.parametrize("kind", ["chain", "tree"])
def test_windows(dev, dt, window, sinks, kind):
    """Short rows and long ones, empty ones, windows narrower than the block and wider than the row."""
    rng = np.random.default_rng(window % 1000 + sinks % 1000)
    for room in (0, 128):
        L.Case(rng, dev, 5, 9, 4, 2, 64, 16, [0, 1, 44, 700, 333], dt, kind, lens=[9, 4, 9, 7, 0], room=room).run(window, sinks)


@pytest.mark.parametrize("dt", L.TYPES)
@pytest.mark.parametrize("T,Hq,H,D", [(1, 32, 8, 128), (17, 8, 2, 128), (33, 4, 1, 128), (70, 2, 1, 64), (64, 6, 2, 256),
                                      (8, 8, 1, 256), (130, 1, 1, 128), (20, 4, 4, 96), (200, 4, 2, 64)])
def test_rows_and_heads(dev, dt, T, Hq, H, D):
    """Every choice of kernel; trees whose depths matter to a narrow window."""
    rng = np.random.default_rng(T + D)
    for window, sinks in ((3, 1), (90, 4)):
        L.Case(rng, dev, 2, T, Hq, H, D, 16, [401, 20], dt, "tree", room=64).run(window, sinks)


@pytest.mark.parametrize("dt", L.TYPES)
def test_any_visibility(dev, dt):
    L.Case(np.random.default_rng(2), dev, 3, 40, 4, 2, 128, 32, [0, 600, 33], dt, "random", room=64).run(6, 2)


@pytest.mark.parametrize("dt", L.TYPES)
@pytest.mark.parametrize("P", [1, 48, 200])
def test_pages(dev, dt, P):
    L.Case(np.random.default_rng(P), dev, 3, 5, 8, 2, 128, P, [255, 64, 900], dt, "chain").run(100, 5)


@pytest.mark.parametrize("dt", L.TYPES)
def test_far_rows(dev, dt):
    """Rows far longer than the window, split over workgroups; sinks in the first rounds alone."""
    L.Case(np.random.default_rng(7), dev, 3, 3, 4, 1, 128, 64, [30000, 9000, 2500], dt, "chain").run(2000, 4)


@pytest.mark.parametrize("dt", L.TYPES)
def test_what_no_node_sees_is_not_looked_at(dev, dt):
    """NaN and page ids that are none, before the window and behind the sinks."""
    c = L.Case(np.random.default_rng(11), dev, 1, 4, 4, 2, 64, 16, [4000], dt, "chain")
    c.run(100, 4)
    out, lse = c.attend(100, 4)
    rows = c.places(c.table_np, 0, np.arange(4, 4000 - 99))
    for t, s in ((c.k, c.k_block), (c.v, c.v_block)):
        if dt is L.BF16:
            t.view(torch.int16)[rows] = 0x7FC0
        elif dt is L.E4M3:
            t.view(torch.uint8)[rows] = 0x7F
        else:
            s.view(torch.uint8)[rows] = 255
    c.table[0, 40:200] = -1     # positions 640 .. 3199
    o2, l2 = c.attend(100, 4)
    torch.cuda.synchronize()
    assert ds.device_error() == 0
    assert torch.equal(out, o2) and torch.equal(lse, l2)


def test_depths_outside_are_held(dev):
    c = L.Case(np.random.default_rng(5), dev, 1, 4, 2, 1, 64, 16, [50], L.BF16, "tree")
    c.depth.copy_(torch.tensor([[-7, 1, 900, 3]], dtype=torch.int32))
    c.depth_np = np.array([[0, 1, 3, 3]])
    c.run(3, 2)


def test_a_window_over_everything_is_tree_attn(dev):
    for dt in L.TYPES:
        c = L.Case(np.random.default_rng(6), dev, 3, 9, 8, 2, 128, 16, [0, 93, 2000], dt, "tree")
        a, b = c.attend(), c.attend(1 << 20, 0)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_captured_and_replayed(dev):
    rng = np.random.default_rng(14)
    c = L.Case(rng, dev, 3, 4, 8, 2, 128, 16, [50, 3000, 0], L.BF16, "chain")
    out, lse = torch.zeros_like(c.q), torch.zeros((3, 4, 8), device=dev)
    c.attend(500, 4, out, lse)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.attend(500, 4, out, lse)
    for i in range(4):
        c.q.copy_(torch.from_numpy(rng.standard_normal(c.q.shape).astype(np.float32)).to(dev))
        c.seq_len.copy_(torch.tensor([50 - i, 3000 - 700 * i, i], dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        got = out.clone(), lse.clone()
        out.zero_(), lse.zero_()
        c.attend(500, 4, out, lse)
        torch.cuda.synchronize()
        # bits: the last row comes to places that hold NaN
        assert torch.equal(got[0].view(torch.int16), out.view(torch.int16)), i
        assert torch.equal(got[1].view(torch.int32), lse.view(torch.int32)), i


@pytest.mark.parametrize("dt", L.TYPES)
def test_many_rows(dev, dt):
    """More rows than a wave has lanes, each with a window of its own place."""
    rng = np.random.default_rng(21)
    L.Case(rng, dev, 150, 2, 4, 2, 64, 16, rng.integers(0, 400, 150), dt, "chain", lens=rng.integers(0, 3, 150)).run(70, 3)


def test_a_window_over_a_mask_alone_and_depths_alone(dev):
    """A mask without depths puts node i at i; depths without a mask leave the chain's visibility."""
    c = L.Case(np.random.default_rng(22), dev, 2, 6, 2, 1, 64, 16, [40, 3], L.BF16, "tree")
    depth, c.depth = c.depth, None
    real, c.depth_np = c.depth_np, np.tile(np.arange(6), (2, 1))
    c.run(3, 1)
    c.depth, c.depth_np, c.mask = depth, real, None
    c.vis = np.tile(np.tril(np.ones((6, 6), bool)), (2, 1, 1))
    c.run(3, 1)
