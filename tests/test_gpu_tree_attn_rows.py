"""tree_attn on the GPU: what a node's result may depend on, down to its bits."""
import numpy as np
import pytest
import torch

import draft_selection_amd as ds
import test_gpu_tree_attn as ta

pytestmark = pytest.mark.gpu
DTYPES = ta.DTYPES


def _bits(o, l):
    return o.view(torch.int16).clone(), l.view(torch.int32).clone()


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("T,Hq,H,D", [(5, 4, 2, 64), (9, 4, 1, 128), (17, 4, 1, 128), (40, 8, 1, 128), (6, 8, 1, 256),
                                      (21, 8, 1, 256)])
@pytest.mark.parametrize("wide", [False, True])
def test_other_queries_change_no_bit(dev, dt, T, Hq, H, D, wide):
    """The queries of other nodes and other heads, whose running maximum moves at other keys, leave a result as it is."""
    rng = np.random.default_rng(T * D)
    q, a, *_ = ta._setup(rng, dev, 2, T, Hq, H, D, 16, [230, 180] if not wide else [3000, 900], dt)
    if wide:
        a = ta._widen(a)
    first = _bits(*ds.tree_attn(q, want_lse=True, **a))
    keep = torch.zeros(q.shape[:3], dtype=torch.bool, device=dev)
    keep[:, ::3, 1] = True                                        # these queries stay, every other one grows
    for factor in (8.0, 60.0, 0.0):
        p = torch.where(keep[..., None], q, (factor * q.float()).to(torch.bfloat16))
        got = _bits(*ds.tree_attn(p, want_lse=True, **a))
        assert torch.equal(got[0][keep], first[0][keep]) and torch.equal(got[1][keep], first[1][keep])
    assert ds.device_error() == 0


@pytest.mark.parametrize("T,G,D", [(7, 4, 64), (40, 2, 128), (33, 4, 128), (9, 8, 256)])
@pytest.mark.parametrize("wide", [False, True])
def test_a_scale_that_is_nan(dev, T, G, D, wide):
    """Nodes that see something under it get NaN, nodes that see nothing 0 and -inf, other heads what they got."""
    rng = np.random.default_rng(T + D)
    q, a, K, V, vis, seq, n = ta._setup(rng, dev, 3, T, 2 * G, 2, D, 16, [0, 5, 0], torch.float8_e4m3fn, kind="random")
    if wide:
        a = ta._widen(a)
    first, l1 = ds.tree_attn(q, want_lse=True, **a)
    a["k_scale"][1] = float("nan")
    out, lse = ds.tree_attn(q, want_lse=True, **a)
    assert torch.equal(out[:, :, :G], first[:, :, :G]) and torch.equal(lse[:, :, :G], l1[:, :, :G])
    blind = torch.from_numpy(~vis.any(2) & (seq == 0)[:, None]).to(dev)
    assert blind.any() and not blind.all()
    assert (out[:, :, G:][blind] == 0).all() and lse[:, :, G:][blind].isneginf().all()
    assert out[:, :, G:][~blind].isnan().all() and lse[:, :, G:][~blind].isnan().all()
