"""Attention whose shares of work go through several rounds of keys, for every choice of kernel: whole tiles of a narrow
window that two or three rounds hold, and long rows of a batch that gives every workgroup more than two rounds (bounds:
longcache.py).  The rows' last rounds end inside, where lanes without a key stand beside lanes with one."""
import numpy as np
import pytest
import torch

import draft_selection_amd as ds
import longcache as L

pytestmark = pytest.mark.gpu


def _repeated(c, times):
    """The batch of ``c`` many times over the same pages, with queries of their own."""
    g = torch.Generator(device=c.dev).manual_seed(c.T)
    c.B, c.K, c.V = c.B * times, c.K * times, c.V * times
    c.seq, c.n, c.depth_np, c.vis = (np.concatenate([x] * times) for x in (c.seq, c.n, c.depth_np, c.vis))
    for name in ("table", "seq_len", "block_len", "mask", "depth"):
        t = getattr(c, name)
        if t is not None:
            setattr(c, name, t.repeat(times, *[1] * (t.dim() - 1)))
    c.q = (2 * torch.randn((c.B, *c.q.shape[1:]), generator=g, device=c.dev)).to(L.BF16)
    return c


def _check(c, window, sinks, rows):
    out, lse = c.attend(window, sinks)
    again = c.attend(window, sinks)
    torch.cuda.synchronize()
    assert ds.device_error() == 0
    c.check(out, lse, window, sinks, rows=rows)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


@pytest.mark.parametrize("dt", L.TYPES)
@pytest.mark.parametrize("D", [64, 96, 128, 160, 256])
@pytest.mark.parametrize("T", [1, 4, 6, 10, 18, 33, 40])     # times 4 heads: every row count that a kernel is chosen by
def test_whole_tiles_of_several_rounds(dev, dt, D, T):
    rng = np.random.default_rng(D + T)
    c = L.Case(rng, dev, 6, T, 8, 2, D, 16, [300, 290, 700, 511, 515, 258], dt, "chain")
    for window, sinks in ((10, 4), (8, 1)):
        _check(c, window, sinks, range(6))


@pytest.mark.parametrize("dt", L.TYPES)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("T", [1, 4, 6, 10, 18, 33])
def test_shares_of_several_rounds(dev, dt, D, T):
    rng = np.random.default_rng(D + T + 1)
    c = L.Case(rng, dev, 5, T, 16, 4, D, 16, [1000, 777, 1290, 640, 1023], dt, "tree", lens=[T, max(1, T // 2), T, T, T], room=128)
    c = _repeated(c, 24)
    for window, sinks in ((None, 0), (900, 4), (300, 0)):
        _check(c, window, sinks, (0, 1, 58, 62, 118))
