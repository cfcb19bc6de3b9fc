"""pages_fork on the GPU where a source row holds a page id that is none."""
import pytest
import torch

import draft_selection_amd as ds

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bad", [-1, 8, 1 << 30])
@pytest.mark.parametrize("at", [0, 2])
def test_fork_of_a_row_with_a_bad_page(dev, bad, at):
    """Positions that no query sees in the source are seen by none in the copy: the id is taken along, whole page or
    partial one, and the page planned for the copy stays free.  Other copies are made."""
    P = 4
    t = lambda *a: torch.tensor(a, dtype=torch.int32, device=dev)
    k = torch.randn((2, 8, P, 1, 8), device=dev).to(torch.bfloat16)
    v = k + 1
    kk, vv = k.clone(), v.clone()
    src = [5, 1, 6]
    src[at] = bad
    p = ds.Pages(torch.tensor([src, [-1] * 3, [3, -1, -1], [-1] * 3], dtype=torch.int32, device=dev), t(3, 0, 1, 0),
                 t(10, 0, 3, 0), t(0, 1, 0, 1, 0, 1, 1, 0), P)
    assert ds.pages_fork(p, t(-1, 0, -1, 2), k, v).tolist() == [1]
    assert ds.device_error() == ds.DEVERR_PAGE
    # planned: page 0 for row 1, page 2 for row 3
    copy = [x if i < 2 else 0 for i, x in enumerate(src)]
    ref = [1, 1, 1, 1, 0, 1, 1, 0]
    for i in (0, 1):
        if src[i] != bad:
            ref[src[i]] += 1
    if at == 2:
        copy[2], ref[0] = bad, 0
    else:
        kk[:, 0, :2], vv[:, 0, :2] = k[:, 6, :2], v[:, 6, :2]
    kk[:, 2, :3], vv[:, 2, :3] = k[:, 3, :3], v[:, 3, :3]
    assert p.table.tolist() == [src, copy, [3, -1, -1], [2, -1, -1]]
    assert p.refcount.tolist() == ref and p.row_pages.tolist() == [3, 3, 1, 1] and p.seq_len.tolist() == [10, 10, 3, 3]
    assert torch.equal(k, kk) and torch.equal(v, vv)
    assert ds.pages_reserve(p, t(0, 0, 0, 2)).tolist() == [1]      # the lowest free page is handed out again
    assert p.table[3].tolist() == [2, 0 if at == 2 else 4, -1] and ds.device_error() == 0
