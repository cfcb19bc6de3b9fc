"""tree_attn on the GPU against the fp64 oracle, and a whole step of the cache side of verification.

Tolerance, derived from the arithmetic (u = 2^-24, h = 2^-8, half a bf16 step
relative to the value).  A score is an fp32 sum of D exact products (error at
most D u sum |q||K| scale in any order) times scale and log2 e, rounded a few
times more; with the subtraction of the maximum and the hardware's exp2 (a few
units in the last place) a weight is off by at most a relative
    e_z = 2 (D + 8) u zmag + 16 u,     zmag = max_j sum |q||K_j| scale,
numerator and denominator alike.  The weights are rounded to bf16 (h) for their
product with V; sums over N keys add N u in any order.  So, with A = sum p |V|,
    |out - ref| <= 1.01 (A (h + 2 e_z + 2 (N + 64) u) + h |ref|),
    |lse - ref| <= 1.01 (e_z + (N + 64) u + 4 u |ref| + 4 u)."""
import numpy as np
import pytest
import torch

import draft_selection_amd as ds
from oracle import tree as ot

pytestmark = pytest.mark.gpu
U, HALF = 2.0 ** -24, 2.0 ** -8
NAN_CODE = {torch.bfloat16: 0x7FC0, torch.float8_e4m3fn: 0x7F}


def _visibility(rng, B, T, kind):
    """(mask bits or None, truth values [B, T, T])."""
    if kind == "chain":
        return None, np.tile(np.tril(np.ones((T, T), bool)), (B, 1, 1))
    if kind == "tree":
        vis = np.stack([ot.ancestors([-1] + [int(rng.integers(max(0, i - 6), i)) for i in range(1, T)])[0] for _ in range(B)])
    elif kind == "all":
        vis = np.ones((B, T, T), bool)
    else:  # "random": any visibility, rows that see nothing among it
        vis = rng.random((B, T, T)) < 0.4
        vis[:, ::3] = False
    return ot.pack(vis), vis


def _setup(rng, dev, B, T, Hq, H, D, P, ctx, dt, kind="tree", layout="tokens", lens=None, q_std=2.0, spare_cols=1):
    """Inputs with NaN in every place that no query may read."""
    seq = np.asarray(ctx, np.int32)
    n = np.full(B, T, np.int32) if lens is None else np.asarray(lens, np.int32)
    cols = int(max((seq + T + P - 1) // P)) + spare_cols
    pages = B * cols + 1
    table = rng.permutation(pages)[:B * cols].reshape(B, cols).astype(np.int32)
    it = torch.int16 if dt == torch.bfloat16 else torch.uint8
    shape = (pages, H, P, D) if layout == "heads" else (pages, P, H, D)
    if layout == "interleaved":
        raw = torch.full((pages, 2, P, H, D), NAN_CODE[dt], dtype=it, device=dev)
        k, v = raw[:, 0].view(dt), raw[:, 1].view(dt)
    else:
        k, v = (torch.full(shape, NAN_CODE[dt], dtype=it, device=dev).view(dt) for _ in range(2))
        if layout == "heads":
            k, v = k.transpose(1, 2), v.transpose(1, 2)
    scales = {}
    if dt == torch.float8_e4m3fn:
        scales = {s: torch.from_numpy(rng.uniform(0.01, 0.03, H).astype(np.float32)).to(dev) for s in ("k_scale", "v_scale")}
    K, V = [], []
    for b in range(B):
        N = int(seq[b] + n[b])
        pos = np.arange(N)
        rows = torch.from_numpy(table[b][pos // P].astype(np.int64)).to(dev), torch.from_numpy(pos % P).to(dev)
        for cache, s, got in ((k, "k_scale", K), (v, "v_scale", V)):
            x = torch.from_numpy(rng.standard_normal((N, H, D)).astype(np.float32)).to(dev)
            if scales:
                x = (x / scales[s][None, :, None]).clamp(-448, 448).to(dt)
                ref = x.double() * scales[s][None, :, None].double()
            else:
                x = x.to(dt)
                ref = x.double()
            cache.view(it)[rows] = x.view(it)
            got.append(ref.cpu().numpy())
    if table.shape[1] > cols - spare_cols:
        for b in range(B):
            table[b, (int(seq[b] + n[b]) + P - 1) // P:] = 1 << 30   # never looked at
    q = torch.from_numpy((q_std * rng.standard_normal((B, T, Hq, D))).astype(np.float32)).to(dev).to(torch.bfloat16)
    bits, vis = _visibility(rng, B, T, kind)
    d = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(dev)
    args = dict(k_cache=k, v_cache=v, page_table=d(table), seq_len=d(seq), mask=None if bits is None else d(bits),
                block_len=None if lens is None else d(n), **scales)
    return q, args, K, V, vis, seq, n


def _check(out, lse, q, K, V, vis, seq, n, scale, rows=None):
    B, T, Hq, D = q.shape
    for b in rows if rows is not None else range(B):
        m, s = int(n[b]), int(seq[b])
        sees = np.ones((m, s + m), bool)
        sees[:, s:] = vis[b, :m, :m]
        ref, rl, mag, zmag = ot.attend(q[b, :m].double().cpu().numpy(), K[b], V[b], sees, scale)
        o, l = out[b, :m].double().cpu().numpy(), lse[b, :m].double().cpu().numpy()
        N = s + m
        ez = 2 * (D + 8) * U * zmag + 16 * U
        tol = 1.01 * (mag * (HALF + 2 * ez + 2 * (N + 64) * U)[..., None] + HALF * np.abs(ref))
        bad = ~(np.abs(o - ref) <= tol + 1e-38)
        assert not bad.any(), (b, np.argwhere(bad)[:4], o[bad][:4], ref[bad][:4], tol[bad][:4])
        fin = np.isfinite(rl)
        assert np.array_equal(np.isneginf(l), np.isneginf(rl))
        tl = 1.01 * (ez + (N + 64) * U + 4 * U * np.abs(np.where(fin, rl, 0)) + 4 * U)
        assert (np.abs(l[fin] - rl[fin]) <= tl[fin]).all()
        assert (o[~fin] == 0).all()


def _widen(args, to=4096):
    """The same table in a wider one: rows that could hold more keys are split over workgroups and joined."""
    t = args["page_table"]
    wide = torch.full((t.shape[0], max(to, t.shape[1])), -9, dtype=torch.int32, device=t.device)
    wide[:, :t.shape[1]] = t
    return {**args, "page_table": wide}


def _run(dev, rng, *shape, **kw):
    """One call with the table as it is, one with room for long rows."""
    q, args, *ref = _setup(rng, dev, *shape, **kw)
    B, T, Hq, D = q.shape
    n = ref[4]
    for a in (args, _widen(args)):
        out = torch.full((B, T, Hq, D), 7.0, dtype=torch.bfloat16, device=dev)
        lse = torch.full((B, T, Hq), 7.0, device=dev)
        ds.tree_attn(q, out=out, lse=lse, **a)
        torch.cuda.synchronize()
        assert ds.device_error() == 0
        _check(out, lse, q, *ref, D ** -0.5)
        for b in range(B):
            assert (out[b, n[b]:] == 7).all() and (lse[b, n[b]:] == 7).all()


DTYPES = [torch.bfloat16, torch.float8_e4m3fn]


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("Hq,H,D", [(1, 1, 128), (4, 1, 128), (10, 2, 128), (8, 8, 64), (16, 2, 256), (3, 3, 80),
                                    (5, 1, 16), (2, 1, 176)])
def test_heads(dev, dt, Hq, H, D):
    rng = np.random.default_rng(Hq * 1000 + D)
    _run(dev, rng, 3, 7, Hq, H, D, 16, [0, 93, 300], dt)


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("P", [1, 5, 16, 48, 64, 200])
@pytest.mark.parametrize("layout", ["tokens", "heads", "interleaved"])
def test_pages_and_layouts(dev, dt, P, layout):
    rng = np.random.default_rng(P)
    _run(dev, rng, 4, 9, 4, 2, 128, P, [P - 1, P, 3 * P + 1, 170], dt, layout=layout)


@pytest.mark.parametrize("kind", ["chain", "tree", "all", "random"])
@pytest.mark.parametrize("T", [1, 2, 8, 17, 31, 32, 33, 60, 64, 65, 129, 256])
def test_tree_sizes_and_masks(dev, kind, T):
    """Row groups of every size the kernel chooses between, masks that leave rows with nothing to see."""
    rng = np.random.default_rng(T)
    lens = [T, 0, max(1, T // 2), T, T]
    _run(dev, rng, 5, T, 4, 2, 64, 16, [0, 40, 0, 65, 129], torch.bfloat16, kind=kind, lens=lens)


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("D,G", [(128, 4), (64, 1), (256, 8), (112, 2)])
@pytest.mark.parametrize("T", [1, 16, 70])
def test_long_rows(dev, dt, D, G, T):
    """Long caches beside short ones: work split along the keys and joined."""
    rng = np.random.default_rng(D + T)
    ctx = [5000, 3, 0, 1023, 1024, 2600]
    _run(dev, rng, 6, T, G, 1, D, 32, ctx, dt, lens=[T, T, T, 1, T, 0], kind="random" if T == 16 else "tree")


@pytest.mark.parametrize("B", [64, 65, 200, 777])
def test_many_rows(dev, B):
    """More rows than a wave has lanes, most of them short, some empty, a few long."""
    rng = np.random.default_rng(B)
    ctx = rng.integers(0, 60, B)
    ctx[rng.integers(0, B, 5)] = rng.integers(500, 3000, 5)
    lens = rng.integers(0, 3, B)
    lens[ctx > 400] = 2
    _run(dev, rng, B, 2, 2, 1, 64, 16, ctx, torch.bfloat16, lens=lens, kind="chain")


@pytest.mark.parametrize("scales", [(0.0, 1.0), (-0.02, -0.5), (0.02, 0.0)])
def test_scales_of_any_sign(dev, scales):
    rng = np.random.default_rng(8)
    q, a, K, V, vis, seq, n = _setup(rng, dev, 2, 6, 4, 1, 64, 16, [90, 33], torch.float8_e4m3fn)
    old = a["k_scale"].item(), a["v_scale"].item()
    K, V = [x * (scales[0] / old[0]) for x in K], [x * (scales[1] / old[1]) for x in V]
    a["k_scale"].fill_(scales[0])
    a["v_scale"].fill_(scales[1])
    K, V = [x * (float(np.float32(scales[0])) / scales[0]) if scales[0] else x for x in K], V
    out, lse = ds.tree_attn(q, want_lse=True, **a)
    _check(out, lse, q, K, V, vis, seq, n, 64 ** -0.5)
    a["k_scale"].fill_(float("nan"))
    assert ds.tree_attn(q, **a)[0].isnan().all()


def test_large_and_small_scores(dev):
    """Scores whose softmax is one key, and scores that are all alike."""
    rng = np.random.default_rng(3)
    _run(dev, rng, 2, 9, 4, 1, 128, 16, [700, 100], torch.bfloat16, q_std=300.0)
    _run(dev, rng, 2, 9, 4, 1, 128, 16, [700, 100], torch.bfloat16, q_std=0.0)


@pytest.mark.parametrize("dt", DTYPES)
def test_scale_strides_and_table_views(dev, dt):
    """q as a slice of a fused projection, a table that is a view, a given scale."""
    rng = np.random.default_rng(5)
    q, a, K, V, vis, seq, n = _setup(rng, dev, 3, 11, 8, 2, 128, 16, [50, 0, 222], dt)
    fused = torch.full((3, 11, 12, 128), float("nan"), dtype=torch.bfloat16, device=dev)
    fused[:, :, 2:10] = q
    table = torch.full((3, a["page_table"].shape[1] + 5), -1, dtype=torch.int32, device=dev)
    table[:, :-5] = a["page_table"]
    a["page_table"] = table[:, :-5]
    out, lse = ds.tree_attn(fused[:, :, 2:10], scale=0.31, want_lse=True, **a)
    _check(out, lse, q, K, V, vis, seq, n, float(np.float32(0.31)))
    by_head = q.permute(2, 0, 1, 3).contiguous().permute(1, 2, 0, 3)
    again, none = ds.tree_attn(by_head, scale=0.31, **a)
    assert none is None and torch.equal(again, out)
    assert ds.device_error() == 0


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("ctx,T,G", [(0, 40, 2), (77, 9, 1), (2000, 33, 4), (30, 100, 4)])
@pytest.mark.parametrize("wide", [False, True])
def test_unseen_infinities_and_nan(dev, dt, ctx, T, G, wide):
    """Nodes with NaN or infinite K and V: nodes that do not see them get what they would get without."""
    rng = np.random.default_rng(ctx + T)
    q, a, K, V, vis, seq, n = _setup(rng, dev, 2, T, G, 1, 64, 16, [ctx, ctx + 3], dt, kind="random")
    vis[:, :, 0] = True                                           # nobody's softmax is empty
    bad = [4, T - 2]
    vis[:, :, bad] &= (np.arange(T) % 2 == 0)[None, :, None]      # odd nodes see none of them
    a["mask"] = torch.from_numpy(ot.pack(vis)).to(dev)
    tab = a["page_table"].cpu().numpy()
    inf = float("inf") if dt == torch.bfloat16 else float("nan")
    for b in range(2):
        for i, j in enumerate(bad):
            p = int(seq[b]) + j
            a["k_cache"][int(tab[b, p // 16]), p % 16] = torch.tensor(float("nan") if i else 1.0, device=dev).to(dt)
            a["v_cache"][int(tab[b, p // 16]), p % 16] = torch.tensor([inf, -inf, float("nan"), 1.0] * 16, device=dev).to(dt)
    if wide:
        a = _widen(a)
    out, lse = ds.tree_attn(q, want_lse=True, **a)
    assert ds.device_error() == 0
    odd = np.zeros_like(vis)
    odd[:, 1::2] = vis[:, 1::2]
    for b in range(2):
        s, m = int(seq[b]), T
        K[b][s + bad[0]], K[b][s + bad[1]], V[b][s + bad[0]], V[b][s + bad[1]] = 0, 0, 0, 0
        sees = np.ones((m, s + m), bool)
        sees[:, s:] = odd[b]
        keep = np.arange(1, T, 2)
        ref, rl, mag, zmag = ot.attend(q[b, keep].double().cpu().numpy(), K[b], V[b], sees[keep], 64 ** -0.5)
        o, l = out[b, keep].double().cpu().numpy(), lse[b, keep].double().cpu().numpy()
        ez = 2 * (64 + 8) * U * zmag + 16 * U
        tol = 1.01 * (mag * (HALF + 2 * ez + 2 * (s + m + 64) * U)[..., None] + HALF * np.abs(ref))
        assert (np.abs(o - ref) <= tol).all()
        assert (np.abs(l - rl) <= 1.01 * (ez + (s + m + 64) * U + 4 * U * np.abs(rl) + 4 * U)).all()
        # the others see what is there: NaN keys make them NaN, infinite values stay infinite
        for i in range(0, T, 2):
            if vis[b, i, bad[1]]:
                assert out[b, i].isnan().all() and lse[b, i].isnan().all()
            elif vis[b, i, bad[0]]:
                o = out[b, i].float().view(G, 16, 4)
                if dt == torch.bfloat16:
                    assert (o[..., 0] == inf).all() and (o[..., 1] == -inf).all()
                assert o[..., 2].isnan().all() and o[..., 3].isfinite().all() and lse[b, i].isfinite().all()


def test_bad_rows_and_pages(dev):
    """Lengths that the table cannot hold make a row empty; a page that is none is seen by nobody."""
    rng = np.random.default_rng(9)
    q, a, K, V, vis, seq, n = _setup(rng, dev, 4, 5, 2, 1, 64, 16, [100, 20, 50, 64], torch.bfloat16, kind="chain")
    a["seq_len"][1] = -1
    a["seq_len"][2] = a["page_table"].shape[1] * 16 - 4
    a["page_table"][3, 1] = -7
    a["page_table"][3, 2] = a["k_cache"].shape[0]
    b = _widen(a)
    b["seq_len"] = a["seq_len"].clone()
    b["seq_len"][2] = b["page_table"].shape[1] * 16 - 4
    for a in (a, b):
        out = torch.full_like(q, 7.0)
        lse = torch.full(q.shape[:3], 7.0, device=dev)
        ds.tree_attn(q, out=out, lse=lse, **a)
        assert ds.device_error() == ds.DEVERR_SEQ_LEN | ds.DEVERR_PAGE
        assert (out[1:3] == 7).all() and (lse[1:3] == 7).all()
        _check(out, lse, q, K, V, vis, seq, n, 64 ** -0.5, rows=[0])
        cut = [np.concatenate([x[3][:16], x[3][48:]]) for x in (K, V)]
        _check(out[3:], lse[3:], q[3:], [cut[0]], [cut[1]], vis[3:], [seq[3] - 32], n[3:], 64 ** -0.5)


def test_offsets_past_32_bits(dev):
    """Pages further than 2^32 bytes into the cache."""
    rng = np.random.default_rng(1)
    q, a, K, V, vis, seq, n = _setup(rng, dev, 2, 9, 8, 2, 128, 64, [300, 77], torch.bfloat16)
    small = a["k_cache"].shape[0]
    per = 64 * 2 * 128
    far = (5 << 30) // (2 * per)                                   # 5 GB of pages in front
    out, _ = ds.tree_attn(q, **a)
    for s in ("k_cache", "v_cache"):
        big = torch.empty((far + small, 64, 2, 128), dtype=torch.bfloat16, device=dev)
        big[far:] = a[s]
        a[s] = big
    cols = (seq + n + 63) // 64
    for b in range(2):
        a["page_table"][b, :cols[b]] += far
    again, _ = ds.tree_attn(q, **a)
    assert torch.equal(out, again) and ds.device_error() == 0
    # the writers' offsets too
    kn = torch.randn((2, 9, 2, 128), device=dev).to(torch.bfloat16)
    ds.cache_append(kn, kn, a["k_cache"], a["v_cache"], a["page_table"], a["seq_len"])
    path = torch.arange(1, 10, dtype=torch.int32, device=dev).repeat(2, 1)
    path[:, 8] = -1
    ds.cache_compact(a["k_cache"], a["v_cache"], a["page_table"], a["seq_len"], path,
                     torch.full((2,), 8, dtype=torch.int32, device=dev))
    tab = a["page_table"].cpu().numpy()
    for b in range(2):
        for i in range(8):
            p = int(seq[b]) + i
            assert torch.equal(a["k_cache"][int(tab[b, p // 64]), p % 64], kn[b, i + 1])
    assert ds.device_error() == 0


def test_same_bits_on_every_call_and_stream(dev):
    """The order of the sums does not change from call to call; calls on two streams at once do not disturb each other."""
    rng = np.random.default_rng(2)
    q, a, *_ = _setup(rng, dev, 3, 20, 8, 2, 128, 16, [9000, 10, 4000], torch.bfloat16)
    first, l1 = ds.tree_attn(q, want_lse=True, **a)
    torch.cuda.synchronize()
    side = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for i in range(6):
        got.append(ds.tree_attn(q, want_lse=True, stream=side[i % 2], **a))
    torch.cuda.synchronize()
    for o, l in got:
        assert torch.equal(o, first) and torch.equal(l, l1)


def test_captured_and_replayed(dev):
    """Two captured calls that share a workspace, one after the other, replayed between eager calls on changed inputs:
    every replay gives what an eager call gives."""
    rng = np.random.default_rng(12)
    q, a, *_ = _setup(rng, dev, 3, 20, 8, 2, 128, 16, [3000, 50, 700], torch.bfloat16)
    q2, a2, *_ = _setup(rng, dev, 2, 40, 8, 1, 64, 16, [600, 900], torch.float8_e4m3fn)
    ws = torch.empty(max(ds.tree_attn_workspace_bytes(3, 20, 8, 2, 128, torch.bfloat16, 1 << 20),
                         ds.tree_attn_workspace_bytes(2, 40, 8, 1, 64, torch.float8_e4m3fn, 1 << 20)),
                     dtype=torch.uint8, device=dev)
    ws.fill_(0xFF)
    outs = [torch.zeros_like(q), torch.zeros_like(q2)]
    graphs = []
    for x, args, o in ((q, a, outs[0]), (q2, a2, outs[1])):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            ds.tree_attn(x, out=o, workspace=ws, **args)
        graphs.append(g)
    for step in range(4):
        q.copy_(torch.randn(q.shape, device=dev).to(torch.bfloat16))
        q2.copy_(torch.randn(q2.shape, device=dev).to(torch.bfloat16))
        if step:
            a["seq_len"] -= 7                                     # a shorter cache: other shares, other joins
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        assert torch.equal(ds.tree_attn(q, **a)[0], outs[0]) and torch.equal(ds.tree_attn(q2, **a2)[0], outs[1])
    assert ds.device_error() == 0


def test_refusals(dev):
    rng = np.random.default_rng(4)
    q, a, *_ = _setup(rng, dev, 2, 5, 4, 2, 64, 16, [30, 9], torch.bfloat16)
    k, v = a["k_cache"], a["v_cache"]
    bad = [dict(q=q.float()), dict(q=q[..., :32]), dict(q=q[:, :, :3]), dict(q=q[0]), dict(k_cache=k.float(), v_cache=v.float()),
           dict(v_cache=v[:, :8]), dict(v_cache=v.transpose(1, 2).contiguous().transpose(1, 2)),
           dict(k_cache=k[None], v_cache=v[None]), dict(page_table=a["page_table"].long()), dict(page_table=a["page_table"][:1]),
           dict(seq_len=a["seq_len"][:1]), dict(mask=a["mask"][:, :4]), dict(mask=a["mask"].long()), dict(scale=0.0),
           dict(scale=float("nan")), dict(k_scale=torch.ones(2, device=dev)), dict(out=torch.empty_like(q)[:1]),
           dict(lse=torch.empty((2, 5, 4), dtype=torch.float64, device=dev)), dict(seq_len=a["seq_len"].cpu()),
           dict(q=q.transpose(1, 3)), dict(block_len=torch.ones(2, dtype=torch.int64, device=dev))]
    for kw in bad:
        b = {"q": q, **a, **kw}
        with pytest.raises((TypeError, ValueError, ds.DselError)):
            ds.tree_attn(b.pop("q"), **b)
    empty, _ = ds.tree_attn(q[:0], k, v, a["page_table"][:0], a["seq_len"][:0])
    assert empty.shape == (0, 5, 4, 64)


# --------------------------------------------------------- a whole step of it ---
def _step(st, new, k_all, v_all, pages, layers):
    """One verification step as a user writes it: tokens' K and V in, attention, the kept path, their rows kept."""
    ds.pages_reserve(pages, st["extra"])
    mask, depth = ds.tree_mask(st["parent"], block_len=st["len"])
    outs = []
    for l in range(layers):
        ds.cache_append(new[0][l], new[1][l], k_all[l], v_all[l], pages.table, pages.seq_len, block_len=st["len"])
        outs.append(ds.tree_attn(st["q"][l], k_all[l], v_all[l], pages.table, pages.seq_len, mask=mask,
                                 block_len=st["len"], out=st["out"][l])[0])
    top = ds.select_topk(st["logits"])[0]
    n_keep, path, out_tok = ds.tree_accept(st["parent"], st["tok"], top[:, :, 0], block_len=st["len"])
    new_len = ds.cache_compact(k_all, v_all, pages.table, pages.seq_len, path, n_keep)
    pages.seq_len.copy_(new_len)
    return outs, n_keep, path, out_tok, depth


@pytest.mark.parametrize("captured", [False, True])
def test_steps_of_verification(dev, captured):
    """Prompts, forks and several steps over three layers, against dense histories kept on the host; also with the
    step captured into a graph and replayed between eager work."""
    rng = np.random.default_rng(11)
    B, T, Hq, H, D, P, L, cols, V = 5, 13, 4, 2, 64, 16, 3, 12, 64
    z = lambda *s: torch.zeros(s, dtype=torch.int32, device=dev)
    pages = ds.Pages(z(B, cols) - 1, z(B), z(B), z(B * cols), P)
    k_all, v_all = (torch.full((L, B * cols, P, H, D), float("nan"), dtype=torch.bfloat16, device=dev) for _ in range(2))
    bf = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32)).to(dev).to(torch.bfloat16)
    hist = [[np.zeros((L, 0, H, D)), np.zeros((L, 0, H, D))] for _ in range(B)]
    # prompts for rows 0..2, then rows 3 and 4 fork from 0 and 2
    first = torch.tensor([37, 16, 50, 0, 0], dtype=torch.int32, device=dev)
    ds.pages_reserve(pages, first)
    kn, vn = bf(L, B, 50, H, D), bf(L, B, 50, H, D)
    ds.cache_append(kn, vn, k_all, v_all, pages.table, pages.seq_len, block_len=first)
    pages.seq_len.copy_(first)
    assert ds.pages_fork(pages, torch.tensor([-1, -1, -1, 0, 2], dtype=torch.int32, device=dev), k_all, v_all).tolist() == [1]
    for b, src in ((0, 0), (1, 1), (2, 2), (3, 0), (4, 2)):
        m = int(first[src])
        hist[b] = [x[:, src, :m].double().cpu().numpy() for x in (kn, vn)]
    st = dict(parent=z(B, T), tok=z(B, T), len=z(B), extra=z(B) + T, q=torch.empty((L, B, T, Hq, D), dtype=torch.bfloat16, device=dev),
              logits=torch.empty((B, T, V), device=dev), out=torch.zeros((L, B, T, Hq, D), dtype=torch.bfloat16, device=dev))
    new = [torch.empty((L, B, T, H, D), dtype=torch.bfloat16, device=dev) for _ in range(2)]

    def draw():
        par = np.stack([[-1] + [int(rng.integers(max(0, i - 4), i)) for i in range(1, T)] for _ in range(B)]).astype(np.int32)
        tok = rng.integers(0, 4, (B, T)).astype(np.int32)
        lens = rng.integers(1, T + 1, B).astype(np.int32)
        lens[int(rng.integers(B))] = 0
        logits = rng.standard_normal((B, T, V)).astype(np.float32)
        logits[:, :, :4] += 3
        for n, a in (("parent", par), ("tok", tok), ("len", lens), ("logits", logits)):
            st[n].copy_(torch.from_numpy(a))
        st["q"].copy_(bf(L, B, T, Hq, D))
        new[0].copy_(bf(L, B, T, H, D))
        new[1].copy_(bf(L, B, T, H, D))
        return par, tok, lens, logits

    graph = res = None
    for step in range(5):
        par, tok, lens, logits = draw()
        before = pages.seq_len.cpu().numpy().copy()
        if captured and step == 1:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                res = _step(st, new, k_all, v_all, pages, L)
        if graph is not None:
            graph.replay()
        else:
            res = _step(st, new, k_all, v_all, pages, L)
        torch.cuda.synchronize()
        outs, n_keep, path, out_tok, depth = res
        assert ds.device_error() == 0
        for b in range(B):
            n, s = int(lens[b]), int(before[b])
            vis, dep = ot.ancestors(par[b, :n])
            for l in range(L):
                Kb = np.concatenate([hist[b][0][l], new[0][l, b, :n].double().cpu().numpy()])
                Vb = np.concatenate([hist[b][1][l], new[1][l, b, :n].double().cpu().numpy()])
                sees = np.ones((n, s + n), bool)
                sees[:, s:] = vis
                ref, _, mag, zmag = ot.attend(st["q"][l, b, :n].double().cpu().numpy(), Kb, Vb, sees, D ** -0.5)
                ez = 2 * (D + 8) * U * zmag + 16 * U
                tol = 1.01 * (mag * (HALF + 2 * ez + 2 * (s + n + 64) * U)[..., None] + HALF * np.abs(ref))
                assert (np.abs(outs[l][b, :n].double().cpu().numpy() - ref) <= tol).all()
            p, o = ot.accept(par[b, :n], tok[b, :n], logits[b].argmax(-1)[:n])
            assert n_keep[b] == len(p) and path[b, :len(p)].tolist() == p and out_tok[b, :len(o)].tolist() == o
            assert int(pages.seq_len[b]) == s + len(p)
            hist[b] = [np.concatenate([h, x[:, b, p].double().cpu().numpy()], 1) for h, x in zip(hist[b], new)]
        # the cache holds the histories
        tab = pages.table.cpu().numpy()
        for b in range(B):
            m = hist[b][0].shape[1]
            pos = np.arange(m)
            for c, h in ((k_all, hist[b][0]), (v_all, hist[b][1])):
                rows = c[:, torch.from_numpy(tab[b][pos // P].astype(np.int64)).to(dev), torch.from_numpy(pos % P).to(dev)]
                assert np.array_equal(rows.double().cpu().numpy(), h)
        ds.tree_mask(st["parent"])                                # eager work between the replays
    ds.pages_free(pages, z(B) + 1)
    assert (pages.refcount == 0).all() and (pages.table == -1).all() and ds.device_error() == 0
