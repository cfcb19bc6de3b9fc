"""Attention over 4-bit caches whose unwritten slots, page 0 among them, hold scale bytes that no call writes: 253 and
254, under which the larger codes pass bf16.  Nothing of a row lies there, so its results are those of its own keys
(bounds: longcache.py)."""
import numpy as np
import pytest
import torch

import draft_selection_amd as ds
import longcache as L

pytestmark = pytest.mark.gpu


def _case(dev, byte, T, Hq, H, D, ctx, lens, room=0, layout="tokens"):
    """A case that does not use page 0, with ``byte`` and codes of 6 and -6 in every slot that it does not use."""
    c = L.Case(np.random.default_rng(T + D + byte), dev, len(ctx), T, Hq, H, D, 16, ctx, L.FP4, "tree", lens=lens, room=room,
               layout=layout)
    raw = [t.view(torch.uint8) for t in (c.k, c.v, c.k_scale, c.v_scale)]
    pages = c.k.shape[0]
    free = sorted(set(range(pages)) - set(c.table_np[(c.table_np >= 0) & (c.table_np < pages)].tolist()))[0]
    if free:
        for t in raw:
            t[free] = t[0]
        c.table_np[c.table_np == 0] = free
        c.table.copy_(torch.from_numpy(c.table_np))
    used = torch.zeros(c.k.shape[:2], dtype=torch.bool, device=dev)
    for b in range(c.B):
        used[c.places(c.table_np, b, np.arange(int(c.seq[b] + c.n[b])))] = True
    assert not used[0].any()
    for t, fill in zip(raw, (0xF7, 0xF7, byte, byte)):
        t[~used] = fill
    return c


# few rows (both tile counts), many rows (rounds of one step and of two), every padded head size
SIZES = [(1, 4, 1, 64), (1, 32, 8, 128), (9, 4, 1, 64), (6, 8, 2, 128), (17, 8, 2, 128), (40, 2, 2, 64), (40, 2, 1, 128),
         (3, 16, 2, 256), (5, 6, 1, 160), (64, 1, 1, 256), (70, 2, 1, 256), (4, 2, 1, 96)]


@pytest.mark.parametrize("byte", [253, 254])
@pytest.mark.parametrize("T,Hq,H,D", SIZES)
def test_slots_of_nobody(dev, byte, T, Hq, H, D):
    for room in (0, 64):
        c = _case(dev, byte, T, Hq, H, D, [0, 93, 130, 45], [T, max(1, T // 2), T, 1], room)
        c.run()
        c.run(20, 3)


@pytest.mark.parametrize("T,Hq,H,D", SIZES)
def test_pages_that_are_none(dev, T, Hq, H, D):
    """A row without one of its pages: its other keys alone count, whatever lies in page 0."""
    c = _case(dev, 254, T, Hq, H, D, [200, 64], [T, max(1, T // 2)], 64, "heads")
    c.table[0, 3], c.table[1, 1] = -1, 1 << 20
    out, lse = c.attend()
    torch.cuda.synchronize()
    assert ds.device_error() == ds.DEVERR_PAGE
    full = c.sees

    def sees(b, window=None, sinks=0):
        m = full(b, window, sinks)
        m[:, (48, 16)[b]:(64, 32)[b]] = False
        return m
    c.sees = sees
    c.check(out, lse)


def test_such_blocks_of_keys_that_a_node_does_not_see(dev):
    """The same bytes in a row's own slots: nodes that do not see the key keep their bits."""
    for T, D in ((6, 128), (40, 64), (40, 256)):
        c = L.Case(np.random.default_rng(T), dev, 1, T, 2, 1, D, 16, [150], L.FP4, "tree", room=64)
        hidden = T - 1
        c.vis[0, :, hidden] = False
        c.mask = L.dev_of(L.ot.pack(c.vis), dev)
        want, wl = (t.clone() for t in c.attend())
        rows = c.places(c.table_np, 0, np.array([150 + hidden]))
        for t, fill in ((c.k, 0xF7), (c.v, 0xF7), (c.k_scale, 254), (c.v_scale, 254)):
            t.view(torch.uint8)[rows] = fill
        out, lse = c.attend()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, wl), (T, D)
    assert ds.device_error() == 0
