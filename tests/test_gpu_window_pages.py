"""tree_attn_window where the pages that no node sees have been given back: every page wholly behind the sinks and before
the window is none, and neither an error is set nor a bit of the result changed; a page that a node sees still sets it."""
import numpy as np
import pytest
import torch

import draft_selection_amd as ds
import longcache as L

pytestmark = pytest.mark.gpu


def _gone(c, b, window, sinks):
    """Pages of row b none of whose positions a node can see."""
    s, m = int(c.seq[b]), int(c.n[b])
    return [i for i in range(-(-(s + m) // c.P)) if i * c.P >= sinks and (i + 1) * c.P <= s - window + 1]


@pytest.mark.parametrize("dt", L.TYPES)
@pytest.mark.parametrize("T,Hq,H,D,P", [(1, 32, 8, 128, 16), (17, 8, 2, 128, 16), (33, 4, 1, 128, 1), (70, 2, 1, 64, 32),
                                        (64, 6, 2, 256, 16), (8, 8, 1, 256, 7), (20, 4, 4, 96, 16), (5, 2, 1, 64, 5),
                                        (200, 2, 1, 64, 64)])
@pytest.mark.parametrize("window,sinks", [(1, 0), (100, 4), (33, 16), (700, 0), (50, 250)])
def test_pages_that_were_given_back(dev, dt, T, Hq, H, D, P, window, sinks):
    rng = np.random.default_rng(T + D + window)
    c = L.Case(rng, dev, 4, T, Hq, H, D, P, [1500, 0, 61, 777], dt, "tree", lens=[T, T, max(1, T // 2), T], room=1600 // P + 300)
    out, lse = c.attend(window, sinks)
    table = c.table_np.copy()
    for b in range(c.B):
        table[b, _gone(c, b, window, sinks)] = (-1, 1 << 30)[b % 2]
    assert (table != c.table_np).any()
    c.table.copy_(torch.from_numpy(table))
    o2, l2 = c.attend(window, sinks)
    torch.cuda.synchronize()
    assert ds.device_error() == 0
    assert torch.equal(out, o2) and torch.equal(lse, l2)
    c.check(o2, l2, window, sinks)


@pytest.mark.parametrize("dt", L.TYPES)
@pytest.mark.parametrize("T,D", [(2, 128), (40, 64), (70, 64)])
def test_pages_that_a_node_sees(dev, dt, T, D):
    """The first page that the root's window reaches, and the last one of the sinks."""
    for page in (0, (900 - 99) // 16):
        c = L.Case(np.random.default_rng(T), dev, 1, T, 2, 1, D, 16, [900], dt, "chain")
        c.table[0, page] = -1
        c.attend(100, 4)
        torch.cuda.synchronize()
        assert ds.device_error() == ds.DEVERR_PAGE, page
    for page in (1, (900 - 99) // 16 - 1):
        c = L.Case(np.random.default_rng(T), dev, 1, T, 2, 1, D, 16, [900], dt, "chain")
        c.table[0, page] = -1
        c.attend(100, 4)
        torch.cuda.synchronize()
        assert ds.device_error() == 0, page
