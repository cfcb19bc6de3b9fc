"""Inputs and bounds for the tests of the long caches' calls, in every cache type.

Bounds, from the arithmetic (u = 2^-24, h = 2^-8, half a bf16 step relative to the
value).  A score is an fp32 sum of D exact products, times scale and log2 e: with
zmag = sum |q||K| scale its error, the subtraction's and the hardware exp2's make a
weight off by a relative e_z = 2 (D + 8) u zmag + 16 u.  Attention: numerator and
denominator alike, weights rounded to bf16 for V, sums over N keys, output rounded:
    |out - ref| <= 1.01 (A (h + 2 e_z + 2 (N + 64) u) + h |ref|),   A = sum p |V|,
    |lse - ref| <= 1.01 (e_z + (N + 64) u + 4 u |ref| + 4 u).
Key weights: the lse enters as given, rounded once as lse log2 e, and count as its
logarithm; a sum of R terms; the decayed sum and the last addition one rounding each:
    |w - ref| <= 1.01 (sum p (2 (D + 8) u zmag + 4 u (|lse| + |ln count| + 8)) + (R + 64) u sum p
                       + 4 u |decay w|)."""
import numpy as np
import torch

import draft_selection_amd as ds
from oracle import longcache as lc
from oracle import tree as ot

U, HALF = 2.0 ** -24, 2.0 ** -8
BF16, E4M3, FP4 = torch.bfloat16, torch.float8_e4m3fn, torch.float4_e2m1fn_x2
TYPES = [BF16, E4M3, FP4]


def dev_of(x, dev):
    return torch.from_numpy(np.ascontiguousarray(x)).to(dev)


def empty_cache(dev, dt, pages, P, H, D, layout="tokens", layers=None):
    """K or V filled with NaN, and its scale bytes (4 bits) or None.  layout: tokens or heads first, or padded rows."""
    lead = () if layers is None else (layers,)
    pad = 32 if layout == "padded" else 0

    def make(n, fill, it):
        if layout == "heads":
            return torch.full((*lead, pages, H, P, n), fill, dtype=it, device=dev).transpose(-3, -2)
        return torch.full((*lead, pages, P, H, n), fill, dtype=it, device=dev)

    if dt is BF16:
        return make(D + pad, 0x7FC0, torch.int16)[..., :D].view(dt), None
    if dt is E4M3:
        return make(D + pad, 0x7F, torch.uint8)[..., :D].view(dt), None
    return (make((D + pad) // 2, 0x5A, torch.uint8)[..., :D // 2].view(FP4),
            make((D + pad) // 32, 255, torch.uint8)[..., :D // 32].view(torch.float8_e8m0fnu))


def put(cache, scale, e4m3_scale, rows, x):
    """Values ``x [N, H, D]`` (numpy) into places ``rows = (pages, slots)``; what they stand for, in fp64."""
    dev = cache.device
    if cache.dtype is BF16:
        t = torch.from_numpy(x.astype(np.float32)).to(dev).to(BF16)
        cache.view(torch.int16)[rows] = t.view(torch.int16)
        return t.double().cpu().numpy()
    if cache.dtype is E4M3:
        t = (torch.from_numpy(x.astype(np.float32)).to(dev) / e4m3_scale[:, None]).clamp(-448, 448).to(E4M3)
        cache.view(torch.uint8)[rows] = t.view(torch.uint8)
        return (t.double() * e4m3_scale.double()[:, None]).cpu().numpy()
    code, byte = lc.to_mxfp4(x)
    cache.view(torch.uint8)[rows] = dev_of(lc.pack(code), dev)
    scale.view(torch.uint8)[rows] = dev_of(byte, dev)
    return lc.from_mxfp4(code, byte)


class Case:
    """A batch: q, caches, table, lengths, a mask; and for each row K, V in fp64 and what each node sees."""

    def __init__(self, rng, dev, B, T, Hq, H, D, P, ctx, dt, kind="tree", layout="tokens", lens=None, q_std=2.0, room=0):
        self.dev, self.B, self.T, self.Hq, self.H, self.D, self.P, self.dt = dev, B, T, Hq, H, D, P, dt
        self.seq = np.asarray(ctx, np.int32)
        self.n = np.full(B, T, np.int32) if lens is None else np.asarray(lens, np.int32)
        cols = int(max((self.seq + T + P - 1) // P))
        pages = B * cols + 1
        table = rng.permutation(pages)[:B * cols].reshape(B, cols).astype(np.int32)
        self.k, self.k_block = empty_cache(dev, dt, pages, P, H, D, layout)
        self.v, self.v_block = empty_cache(dev, dt, pages, P, H, D, layout)
        self.k_scale, self.v_scale = self.k_block, self.v_block
        if dt is E4M3:
            self.k_scale, self.v_scale = (torch.from_numpy(rng.uniform(0.01, 0.03, H).astype(np.float32)).to(dev) for _ in range(2))
        self.K, self.V = [], []
        for b in range(B):
            N = int(self.seq[b] + self.n[b])
            rows = self.places(table, b, np.arange(N))
            for c, blk, s, got in ((self.k, self.k_block, self.k_scale, self.K), (self.v, self.v_block, self.v_scale, self.V)):
                got.append(put(c, blk, s, rows, rng.standard_normal((N, H, D))))
            table[b, (N + P - 1) // P:] = 1 << 30   # never looked at
        if room:
            wide = np.full((B, max(room, cols)), -9, np.int32)
            wide[:, :cols] = table
            table = wide
        self.table_np = table
        self.table, self.seq_len = dev_of(table, dev), dev_of(self.seq, dev)
        self.block_len = None if lens is None else dev_of(self.n, dev)
        self.q = torch.from_numpy((q_std * rng.standard_normal((B, T, Hq, D))).astype(np.float32)).to(dev).to(BF16)
        self.mask = self.depth = None
        self.depth_np = np.tile(np.arange(T), (B, 1))
        if kind == "chain":
            vis = np.tile(np.tril(np.ones((T, T), bool)), (B, 1, 1))
        elif kind == "tree":
            both = [ot.ancestors([-1] + [int(rng.integers(max(0, i - 6), i)) for i in range(1, T)]) for _ in range(B)]
            vis, self.depth_np = np.stack([x[0] for x in both]), np.stack([x[1] for x in both])
        else:  # any visibility, rows that see nothing among it
            vis = rng.random((B, T, T)) < 0.4
            vis[:, ::3] = False
        if kind != "chain":
            self.mask, self.depth = dev_of(ot.pack(vis), dev), dev_of(self.depth_np.astype(np.int32), dev)
        self.vis = vis

    def places(self, table, b, pos):
        return (torch.from_numpy(table[b][pos // self.P].astype(np.int64)).to(self.dev),
                torch.from_numpy(pos % self.P).to(self.dev))

    def sees(self, b, window=None, sinks=0):
        m, s = int(self.n[b]), int(self.seq[b])
        out = np.ones((m, s + m), bool)
        out[:, s:] = self.vis[b, :m, :m]
        return out if window is None else lc.window_sees(out, s, self.depth_np[b, :m], window, sinks)

    def attend(self, window=None, sinks=0, out=None, lse=None, stream=None, **kw):
        B, T, Hq, D = self.q.shape
        out = torch.full((B, T, Hq, D), 7.0, dtype=BF16, device=self.dev) if out is None else out
        lse = torch.full((B, T, Hq), 7.0, device=self.dev) if lse is None else lse
        a = dict(mask=self.mask, block_len=self.block_len, k_scale=self.k_scale, v_scale=self.v_scale, out=out, lse=lse,
                 stream=stream, **kw)
        if window is None:
            return ds.tree_attn(self.q, self.k, self.v, self.table, self.seq_len, **a)
        return ds.tree_attn_window(self.q, self.k, self.v, self.table, self.seq_len, window, sinks=sinks, depth=self.depth, **a)

    def check(self, out, lse, window=None, sinks=0, rows=None):
        scale = self.D ** -0.5
        for b in rows if rows is not None else range(self.B):
            m = int(self.n[b])
            sees = self.sees(b, window, sinks)
            ref, rl, mag, zmag = ot.attend(self.q[b, :m].double().cpu().numpy(), self.K[b], self.V[b], sees, scale)
            o, l = out[b, :m].double().cpu().numpy(), lse[b, :m].double().cpu().numpy()
            N = sees.sum(1).max(initial=0)
            ez = 2 * (self.D + 8) * U * zmag + 16 * U
            tol = 1.01 * (mag * (HALF + 2 * ez + 2 * (N + 64) * U)[..., None] + HALF * np.abs(ref))
            bad = ~(np.abs(o - ref) <= tol + 1e-38)
            assert not bad.any(), (b, np.argwhere(bad)[:4], o[bad][:4], ref[bad][:4], tol[bad][:4])
            fin = np.isfinite(rl)
            assert np.array_equal(np.isneginf(l), np.isneginf(rl))
            tl = 1.01 * (ez + (N + 64) * U + 4 * U * np.abs(np.where(fin, rl, 0)) + 4 * U)
            assert (np.abs(l[fin] - rl[fin]) <= tl[fin]).all()
            assert (o[~fin] == 0).all()
            assert (out[b, m:] == 7).all() and (lse[b, m:] == 7).all()

    def run(self, window=None, sinks=0):
        out, lse = self.attend(window, sinks)
        torch.cuda.synchronize()
        assert ds.device_error() == 0
        self.check(out, lse, window, sinks)


def check_weights(case, got, before, lse, decay, count=None):
    """``got``, ``before [B, n]`` and ``lse [B, T, Hq]`` as numpy fp64."""
    R = case.T * case.Hq
    for b in range(case.B):
        m, s = int(case.n[b]), int(case.seq[b])
        if m == 0:
            assert np.array_equal(got[b], before[b], equal_nan=True)
            continue
        cnt = None if count is None else count[b, :m]
        q = case.q[b, :m].double().cpu().numpy()
        ref, mag = lc.key_weights(q, lse[b, :m], case.K[b][:s], case.D ** -0.5, cnt)
        big = np.abs(np.where(np.isfinite(lse[b, :m]), lse[b, :m], 0)).max(initial=0)
        logc = 0.0 if cnt is None else np.abs(np.log(cnt[cnt > 0])).max(initial=0)
        tol = 1.01 * (2 * (case.D + 8) * U * mag + ref * (4 * U * (big + logc + 8) + (R + 64) * U)) + 1e-37
        want = ref if decay == 0 else decay * before[b, :s] + ref
        if decay:
            tol = tol + 4 * U * np.abs(decay * before[b, :s])
        bad = ~(np.abs(got[b, :s] - want) <= tol)
        assert not bad.any(), (b, np.argwhere(bad)[:4], got[b, :s][bad][:4], want[bad][:4], tol[bad][:4])
        assert np.array_equal(got[b, s:], before[b, s:], equal_nan=True)
