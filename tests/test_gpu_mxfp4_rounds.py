"""Attention over 4-bit caches, where a share of the work has several rounds and some of a workgroup's waves have no
rows: the tiles in LDS change hands in every round, from the first one on (bounds: longcache.py)."""
import numpy as np
import pytest
import torch

import longcache as L

pytestmark = pytest.mark.gpu


def _run(c, window):
    out, lse = c.attend(window, 3)
    for _ in range(4):
        again = c.attend(window, 3)
        torch.cuda.synchronize()
        assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
    assert L.ds.device_error() == 0
    c.check(out, lse, window, 3)


# rounds of 32 keys a wave (33 to 64 rows, and head sizes past 128) beside those of 64
KINDS = [(64, 40, 1), (128, 40, 1), (128, 64, 1), (256, 40, 1), (256, 70, 1), (64, 33, 4), (128, 33, 4)]


@pytest.mark.parametrize("D,T,group", KINDS)
@pytest.mark.parametrize("window", [None, 150])
def test_whole_rows(dev, D, T, group, window):
    """Short tables: a workgroup goes through all rounds of a row, of which the keys have little in common (the scores'
    standard deviation is 4, so that a handful of them decide)."""
    rng = np.random.default_rng(D + T)
    B = 12
    lens = [T, 1, T // 2, 3, T - 1, 0, T, 5, T // 4, 33, 32, 2]
    _run(L.Case(rng, dev, B, T, 2 * group, 2, D, 16, rng.integers(100, 250 - T, B), L.FP4, "tree", lens=lens, q_std=4.0), window)


@pytest.mark.parametrize("D,T,group", KINDS)
@pytest.mark.parametrize("window", [None, 500])
def test_shares_of_several_rounds(dev, D, T, group, window):
    """Divided rows: every share begins in the middle of one, and the next piece of work follows the last in the same tiles."""
    rng = np.random.default_rng(D + T + 1)
    B = 60
    lens = rng.choice([1, 2, 5, T // 3, T - 2, T], B)
    top = 450 if D > 128 else 900
    _run(L.Case(rng, dev, B, T, 2 * group, 2, D, 16, rng.integers(top // 2, top, B), L.FP4, "chain", lens=lens, q_std=4.0,
                room=64), window)
