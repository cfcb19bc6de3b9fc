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


SHAPES = [(1, 4, 1, 128), (7, 4, 2, 64), (17, 4, 1, 128), (40, 8, 1, 80), (21, 8, 1, 256)]


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("T,Hq,H,D", SHAPES)
@pytest.mark.parametrize("wide", [False, True])
def test_other_contents_change_no_bit(dev, dt, T, Hq, H, D, wide):
    """Other rows' queries, keys and masks, the nodes that a node does not see, and where the pages lie: with the same
    lengths none of them changes a result."""
    rng = np.random.default_rng(T + D)
    B, P, it = 3, 16, torch.int16 if dt == torch.bfloat16 else torch.uint8
    q, a, _, _, vis, seq, n = ta._setup(rng, dev, B, T, Hq, H, D, P, [2000, 77, 900] if wide else [190, 77, 0], dt,
                                        lens=[T, max(1, T - 2), T], kind="random")
    if wide:
        a = ta._widen(a)
    first = _bits(*ds.tree_attn(q, want_lse=True, **a))
    tab = a["page_table"].cpu().numpy()
    k, v = a["k_cache"].view(it), a["v_cache"].view(it)
    for row in range(B):
        # every other row: new queries, new keys of ordinary size, no mask bit as it was
        p, b = q.clone(), dict(a)
        kk, vv = k.clone(), v.clone()
        for r in range(B):
            if r != row:
                p[r] = (5 * torch.randn(q[r].shape, device=dev)).to(torch.bfloat16)
                ids = torch.from_numpy(tab[r, :(seq[r] + n[r] + P - 1) // P].astype(np.int64)).to(dev)
                kk[ids], vv[ids] = (torch.randn(kk[ids].shape, device=dev).to(dt).view(it) for _ in range(2))
        b["mask"] = ~a["mask"]
        b["mask"][row] = a["mask"][row]
        # and in the row itself, the nodes that node t does not see
        t = int(rng.integers(n[row]))
        for j in np.nonzero(~vis[row, t, :n[row]])[0]:
            at = tab[row, (seq[row] + j) // P], (seq[row] + j) % P
            kk[at], vv[at] = (torch.randn(kk[at].shape, device=dev).to(dt).view(it) for _ in range(2))
        # the pages in another order
        order = torch.from_numpy(rng.permutation(len(kk))).to(dev)
        b["k_cache"], b["v_cache"] = torch.empty_like(kk), torch.empty_like(vv)
        b["k_cache"][order], b["v_cache"][order] = kk, vv
        b["k_cache"], b["v_cache"] = b["k_cache"].view(dt), b["v_cache"].view(dt)
        inside = (a["page_table"] >= 0) & (a["page_table"] < len(kk))
        b["page_table"] = torch.where(inside, order[a["page_table"].clamp(0, len(kk) - 1).long()].int(), a["page_table"])
        got = _bits(*ds.tree_attn(p, want_lse=True, **b))
        assert torch.equal(got[0][row, t], first[0][row, t]) and torch.equal(got[1][row, t], first[1][row, t])
    assert ds.device_error() == 0


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("T,Hq,H,D", SHAPES)
def test_a_row_alone(dev, dt, T, Hq, H, D):
    """Undivided rows get the bits that they get alone at the same block; divided ones the same to rounding."""
    rng = np.random.default_rng(T * 3 + D)
    for ctx, whole in (([200, 9, 0, 120], True), ([3000, 9, 0, 700], False)):
        ctx = [min(c, 240 - T) for c in ctx] if whole else ctx
        q, a, *ref = ta._setup(rng, dev, 4, T, Hq, H, D, 16, ctx, dt, lens=[T, 1, T, T - T // 3], spare_cols=0)
        n = ref[4]
        cap = a["page_table"].shape[1] * 16
        assert (ds.tree_attn_workspace_bytes(4, T, Hq, H, D, dt, cap) == 0) == whole
        out, lse = ds.tree_attn(q, want_lse=True, **a)
        ta._check(out, lse, q, *ref, D ** -0.5)
        for b in range(4):
            one = {**a, **{k: a[k][b:b + 1] for k in ("page_table", "seq_len", "mask", "block_len")}}
            o, l = ds.tree_attn(q[b:b + 1], want_lse=True, **one)
            K, V, vis, seq, _ = (r[b:b + 1] for r in ref)
            ta._check(o, l, q[b:b + 1], K, V, vis, seq, n[b:b + 1], D ** -0.5)
            if whole:
                assert torch.equal(o[0, :n[b]], out[b, :n[b]]) and torch.equal(l[0, :n[b]], lse[b, :n[b]])
        assert ds.device_error() == 0


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("T,Hq,H,D", SHAPES)
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("q_std", [0.0, 2.0, 200.0])
def test_infinities_and_nan_that_are_seen(dev, dt, T, Hq, H, D, wide, q_std):
    """In cached positions, whose weights are of every size, 0 among them, and among the nodes: a NaN in V makes its
    element NaN, an infinity makes it infinite or NaN, and the other elements stay what they are."""
    rng = np.random.default_rng(T + D)
    q, a, K, V, vis, seq, n = ta._setup(rng, dev, 2, T, Hq, H, D, 16, [2000, 300] if wide else [200, 0], dt, kind="all",
                                        q_std=q_std)
    if wide:
        a = ta._widen(a)
    tab = a["page_table"].cpu().numpy()
    inf = float("inf") if dt == torch.bfloat16 else float("nan")
    plain = torch.arange(D, device=dev) % 4 == 3
    for b in range(2):
        for p in {5 % (seq[b] + T), seq[b] // 2, seq[b] + T // 2}:
            at = int(tab[b, p // 16]), p % 16
            x = a["v_cache"][at].float()
            x[:, 0::4], x[:, 1::4], x[:, 2::4] = inf, -inf, float("nan")
            a["v_cache"][at] = x.to(dt)
    out, lse = ds.tree_attn(q, want_lse=True, **a)
    assert out[..., 2::4].isnan().all() and not out[..., 0::4].isfinite().any() and not out[..., 1::4].isfinite().any()
    if dt == torch.bfloat16:
        assert not (out[..., 0::4] == -inf).any() and not (out[..., 1::4] == inf).any()
    cols = np.arange(D) % 4 == 3
    keep = lambda x: np.where(cols, x, 0.0)
    ta._check(torch.where(plain, out, 0), lse, q, K, [keep(v) for v in V], vis, seq, n, D ** -0.5)
    assert ds.device_error() == 0


@pytest.mark.parametrize("T,Hq,H,D", SHAPES)
@pytest.mark.parametrize("wide", [False, True])
def test_scores_of_minus_infinity(dev, T, Hq, H, D, wide):
    """Keys whose scores are -inf have no weight; a node that sees only such gets 0 and -inf, whatever their V."""
    rng = np.random.default_rng(T)
    q, a, K, V, vis, seq, n = ta._setup(rng, dev, 2, T, Hq, H, D, 16, [700, 900] if wide else [130, 150], torch.bfloat16,
                                        kind="chain")
    if wide:
        a = ta._widen(a)
    q[..., 0] = q[..., 0].abs() + 1
    tab = a["page_table"].cpu().numpy()

    def put(b, p):
        a["k_cache"][int(tab[b, p // 16]), p % 16, :, 0] = -float("inf")
    gone = np.sort(rng.permutation(seq[1] + T)[:(seq[1] + T) // 2])
    for p in range(seq[0] + T):
        put(0, p)
    for p in gone:
        put(1, int(p))
    a["v_cache"][int(tab[0, 0]), 3] = float("inf")
    a["v_cache"][int(tab[0, (seq[0] + T - 1) // 16]), (seq[0] + T - 1) % 16] = float("nan")
    out, lse = ds.tree_attn(q, want_lse=True, **a)
    assert (out[0] == 0).all() and lse[0].isneginf().all()
    left = np.ones(seq[1] + T, bool)
    left[gone] = False
    for t in range(T):
        m = left.copy()
        m[seq[1] + t + 1:] = False
        if m.any():
            ta._check(out[1:, t:t + 1], lse[1:, t:t + 1], q[1:, t:t + 1], [K[1][m]], [V[1][m]], np.ones((1, 1, 1), bool),
                      [int(m.sum()) - 1], [1], D ** -0.5)
    assert ds.device_error() == 0


@pytest.mark.parametrize("T,Hq,H,D", SHAPES)
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("key", [float("inf"), float("nan")])
def test_scores_of_infinity_or_nan(dev, T, Hq, H, D, wide, key):
    """One cached key of one K/V head with such a score: the nodes of its row and its heads get NaN, all else is as it was."""
    rng = np.random.default_rng(T)
    q, a, *_ = ta._setup(rng, dev, 2, T, Hq, H, D, 16, [2500, 900] if wide else [130, 150], torch.bfloat16)
    if wide:
        a = ta._widen(a)
    q[..., 0] = q[..., 0].abs() + 1
    first, l1 = ds.tree_attn(q, want_lse=True, **a)
    at = 40 if not wide else 333
    a["k_cache"][int(a["page_table"][0, at // 16]), at % 16, 0, 0] = key
    out, lse = ds.tree_attn(q, want_lse=True, **a)
    G = Hq // H
    assert out[0, :, :G].isnan().all() and lse[0, :, :G].isnan().all()
    assert torch.equal(out[0, :, G:], first[0, :, G:]) and torch.equal(lse[0, :, G:], l1[0, :, G:])
    assert torch.equal(out[1], first[1]) and torch.equal(lse[1], l1[1]) and ds.device_error() == 0


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("Hq,H,D", [(4, 1, 128), (8, 2, 128), (4, 1, 112), (8, 2, 80), (16, 2, 64), (8, 1, 176), (16, 2, 256)])
@pytest.mark.parametrize("T", [1, 8, 9, 16, 17, 25, 32, 33, 64])
def test_every_count_of_rows(dev, dt, Hq, H, D, T):
    """Nodes times heads of a K/V head on both sides of every number that the kernel chooses by (32, 64, 128, 256), long
    rows beside short ones, against the oracle."""
    rng = np.random.default_rng(T * D + Hq)
    ta._run(dev, rng, 4, T, Hq, H, D, 16, [1500, 0, 61, 300], dt, lens=[T, T, max(1, T - 1), T],
            kind=["tree", "random", "chain"][T % 3])
    ta._run(dev, rng, 3, T, Hq, H, D, 32, [150, 0, 97], dt, kind="random")


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("T,Hq,H,D", SHAPES + [(33, 4, 1, 128), (16, 2, 1, 64), (70, 2, 1, 112)])
@pytest.mark.parametrize("wide", [False, True])
def test_unseen_infinities_and_nan_at_every_head_size(dev, dt, T, Hq, H, D, wide):
    """Nodes that do not see a key get the same bits whether its K and V are numbers, infinities or NaN."""
    rng = np.random.default_rng(T * D)
    q, a, _, _, vis, seq, n = ta._setup(rng, dev, 2, T, Hq, H, D, 16, [900, 2001] if wide else [40, 77], dt, kind="random")
    if wide:
        a = ta._widen(a)
    first = _bits(*ds.tree_attn(q, want_lse=True, **a))
    tab = a["page_table"].cpu().numpy()
    bad = sorted({0, T // 2, T - 1})
    for b in range(2):
        for i, j in enumerate(bad):
            at = int(tab[b, (seq[b] + j) // 16]), (seq[b] + j) % 16
            a["k_cache"][at] = torch.tensor([float("nan"), float("inf"), 1.0][i % 3], device=dev).to(dt)
            a["v_cache"][at] = torch.tensor([float("inf"), -float("inf"), float("nan"), 448.0], device=dev).repeat(D // 4).to(dt)
    got = _bits(*ds.tree_attn(q, want_lse=True, **a))
    blind = torch.from_numpy(~vis[:, :, bad].any(2)).to(dev)
    assert blind.any() or T < 2
    assert torch.equal(got[0][blind], first[0][blind]) and torch.equal(got[1][blind], first[1][blind])
    assert ds.device_error() == 0


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("scale", [1e-45, 1e-38, 2.0 ** 127])
@pytest.mark.parametrize("wide", [False, True])
def test_smallest_and_largest_scale(dev, dt, scale, wide):
    """Scales at the ends of what is taken: queries of zeros (scores of 0 at any scale), and ordinary ones at the small end, where
    the scores are 0 to rounding; nodes with masked keys among them, and nodes that see nothing."""
    rng = np.random.default_rng(7)
    q, a, K, V, vis, seq, n = ta._setup(rng, dev, 2, 9, 4, 1, 64, 16, [0, 900] if wide else [0, 90], dt, kind="random",
                                        q_std=0.0 if scale > 1 else 2.0)
    if wide:
        a = ta._widen(a)
    out, lse = ds.tree_attn(q, scale=scale, want_lse=True, **a)
    ta._check(out, lse, q, K, V, vis, seq, n, float(np.float32(scale)))
    assert ds.device_error() == 0
