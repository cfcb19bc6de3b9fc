"""key_weights where its inputs lie in the gaps of the weights' rows: no memory is shared, and nothing is refused."""
import numpy as np
import pytest
import torch

import draft_selection_amd as ds
import longcache as L

pytestmark = pytest.mark.gpu


def test_inputs_between_rows(dev):
    c = L.Case(np.random.default_rng(0), dev, 3, 2, 4, 2, 64, 16, [50, 40, 20], L.BF16, "chain")
    out, lse = c.attend()
    B, cols = c.table.shape
    n = cols * 16
    want = torch.zeros((B, n), device=dev)
    ds.key_weights(c.q, lse, c.k, c.table, c.seq_len, want)
    slab = torch.full((B, n + 64), -7.0, device=dev)
    w, gap = slab[:, :n], slab[:, n:]
    w.zero_()
    table = gap[:, :cols].view(torch.int32)
    table.copy_(c.table)
    seq, near = gap[0, 40:43].view(torch.int32), gap[1, 16:16 + lse.numel()].view(lse.shape)
    seq.copy_(c.seq_len)
    near.copy_(lse)
    count = gap[2, 50:56].view(B, 2)
    count.fill_(1.0)
    was = slab.clone()
    got = ds.key_weights(c.q, near, c.k, table, seq, w, count=count)
    torch.cuda.synchronize()
    assert ds.device_error() == 0
    # a count of 1 leaves the lse as it is
    assert torch.equal(got, want) and torch.equal(slab[:, n:].view(torch.int32), was[:, n:].view(torch.int32))
    # from the last value of a row on: refused
    for bad in (dict(lse=slab[1, n - 1:n - 1 + lse.numel()].view(lse.shape)), dict(seq_len=slab[0, n - 1:n + 2].view(torch.int32)),
                dict(count=slab[2, n - 3:n + 3].view(B, 2))):
        a = dict(dict(lse=near, seq_len=seq, count=count), **bad)
        with pytest.raises(ds.DselError):
            ds.key_weights(c.q, a["lse"], c.k, table, a["seq_len"], w, count=a["count"])
