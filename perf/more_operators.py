"""Caches that are too long to hold or to read as they are, as they are measured.

Five operators, each in its plain form (elementary torch operations) and as the library's calls:

  attn4    attention of drafted tokens over a paged K/V cache held in 4 bits (tree_attn on such a cache)
  append4  new tokens' rows written into a cache held in 4 bits (cache_append)
  window   attention under a sliding window with a few first positions that stay visible (tree_attn_window)
  weights  the attention weight that every cached position gets, accumulated (key_weights)
  evict    the positions of least weight given up, the others moved together in pages of their own (cache_evict)

The 4-bit format: a block of 32 values along the head dim shares a power of two 2^e, and a value is one of 0, 0.5,
1, 1.5, 2, 3, 4, 6 times that, with a sign; two codes a byte, the first in the low bits, and e + 127 in a byte of its
own.  e is the least whole number with max |x| <= 7 * 2^e.

Every pass leaves a state from which the same pass gives the same outputs.
"""
import math

import torch

own = False
DEV = "cuda"
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------ cases ---
def _attn4(name, B, T, ctx, heads, kv_heads, dim, page, tree=True, ragged=True, layout="heads"):
    c = dict(op="attn4", B=B, T=T, ctx=ctx, heads=heads, kv_heads=kv_heads, dim=dim, page=page, cache="mxfp4", tree=tree,
             ragged=ragged, layout=layout)
    return dict(c, name=name) if name else c


def _append4(name, B, T, ctx, layers, kv_heads, dim, page, ragged=True):
    c = dict(op="append4", B=B, T=T, ctx=ctx, layers=layers, kv_heads=kv_heads, dim=dim, page=page, cache="mxfp4",
             ragged=ragged, layout="heads")
    return dict(c, name=name) if name else c


def _window(name, B, T, ctx, window, sinks, heads, kv_heads, dim, page, cache="bf16", tree=False, ragged=True):
    c = dict(op="window", B=B, T=T, ctx=ctx, window=window, sinks=sinks, heads=heads, kv_heads=kv_heads, dim=dim,
             page=page, cache=cache, tree=tree, ragged=ragged, layout="tokens")
    return dict(c, name=name) if name else c


def _weights(name, B, T, ctx, heads, kv_heads, dim, page, cache="bf16", decay=0.0, ragged=True):
    c = dict(op="weights", B=B, T=T, ctx=ctx, heads=heads, kv_heads=kv_heads, dim=dim, page=page, cache=cache,
             decay=decay, ragged=ragged, layout="tokens")
    return dict(c, name=name) if name else c


def _evict(name, B, ctx, budget, sinks, recent, layers, kv_heads, dim, page):
    c = dict(op="evict", B=B, T=1, ctx=ctx, budget=budget, sinks=sinks, recent=recent, layers=layers, kv_heads=kv_heads,
             dim=dim, page=page, cache="bf16", ragged=True, layout="tokens")
    return dict(c, name=name) if name else c


def listed():
    return [
        # one sequence, one token, a short cache: plain decoding between drafts, where latency counts
        _attn4("attn4_one_token", 1, 1, 333, 32, 8, 128, 16, tree=False, ragged=False),
        # the batched throughput shape: 64 blocks of 16 and the verified token, as chains
        _attn4("attn4_chain17", 64, 17, 4096, 32, 8, 128, 32, tree=False),
        # long prompts kept for decoding, one token each: nothing but reading the cache
        _attn4("attn4_decode_long", 16, 1, 60000, 32, 8, 128, 64, tree=False),
        # one layer's drafted tokens at a small batch, and four prompts of up to 2,048 tokens in eight layers
        _append4("append4_draft", 8, 9, 500, 1, 8, 128, 16),
        _append4("append4_prompt", 4, 2048, 16, 8, 8, 128, 64),
        # a drafter's own narrow window, one sequence: latency
        _window("window_one", 1, 9, 3000, 128, 4, 32, 8, 128, 16, ragged=False),
        # layers with a window of 1,024 in the batched shape, the cache far longer
        _window("window_chain17", 64, 17, 16384, 1024, 4, 32, 8, 128, 32),
        # trees under a window of 4,096 over long caches in 8 bits
        _window("window_tree64_e4m3", 8, 64, 40000, 4096, 4, 32, 8, 128, 64, cache="e4m3", tree=True),
        # one sequence after a token: latency; and what a step of a batch adds to the running sums
        _weights("weights_one_token", 1, 1, 700, 32, 8, 128, 16, ragged=False),
        _weights("weights_chain9", 32, 9, 8192, 32, 8, 128, 32, decay=1.0),
        # a batch cut to half of its length, in all of eight layers
        _evict("evict_layers", 16, 4096, 1500, 4, 256, 8, 8, 128, 32),
        # one short sequence, one layer
        _evict("evict_small", 2, 1100, 512, 4, 64, 1, 8, 128, 16),
    ]


def _span(rng, lo, hi):
    """A whole number of [lo, hi], its logarithm uniform."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    top = {}
    for c in listed():
        w = work(c)
        for k in w:
            top[c["op"], k] = max(top.get((c["op"], k), 0), w[k])
    while True:
        op = rng.choice(["attn4", "attn4", "append4", "window", "window", "weights", "evict"])
        kv = rng.choice([1, 2, 4, 8])
        heads, dim = kv * rng.choice([1, 2, 4, 5, 8]), rng.choice([64, 80, 128, 128, 128, 256])
        page, cache = rng.choice([8, 16, 32, 48, 64, 128]), rng.choice(["bf16", "bf16", "e4m3", "mxfp4"])
        ragged, tree = rng.random() < 0.7, rng.random() < 0.5
        if dim == 80 and (op in ("attn4", "append4") or cache == "mxfp4"):
            dim = rng.choice([32, 96, 160])
        if op == "attn4":
            c = _attn4(None, _span(rng, 1, 64), _span(rng, 1, 100 if tree else 33), _span(rng, 1, 60000), heads, kv, dim,
                       page, tree, ragged, rng.choice(["heads", "tokens"]))
        elif op == "append4":
            c = _append4(None, _span(rng, 1, 64), _span(rng, 1, 1500), _span(rng, 1, 800), _span(rng, 1, 16), kv, dim, page,
                         ragged)
        elif op == "window":
            c = _window(None, _span(rng, 1, 64), _span(rng, 1, 64), _span(rng, 1, 40000), _span(rng, 1, 8000),
                        rng.choice([0, 1, 4, 17]), heads, kv, dim, page, cache, tree, ragged)
        elif op == "weights":
            c = _weights(None, _span(rng, 1, 32), _span(rng, 1, 33), _span(rng, 1, 30000), heads, kv, dim, page, cache,
                         rng.choice([0.0, 0.5, 1.0]), ragged)
        else:
            ctx = _span(rng, 8, 20000)
            sinks, recent = rng.choice([0, 1, 4]), rng.choice([0, 1, 32])
            c = _evict(None, _span(rng, 1, 32), ctx, sinks + recent + _span(rng, 1, ctx), sinks, recent,
                       _span(rng, 1, 16), kv, dim, page)
        w = work(c)
        if all(w[k] <= top[op, k] for k in w) and _held(c) < 4e9:
            return c


def _size(c):
    """Bytes of one value of a case's cache."""
    return {"bf16": 2.0, "e4m3": 1.0, "mxfp4": 17 / 32}[c["cache"]]


def _held(c):
    """Bytes of the caches (both operands) that a case holds, in 16 bits, as its inputs are made."""
    n = c["B"] * (c["ctx"] + c["T"] + c["page"] + c.get("budget", 0))
    return 2 * c.get("layers", 1) * n * c["kv_heads"] * c["dim"] * 2


def _spread(n, lo, hi):
    """n lengths from lo to hi, evenly."""
    return [lo + (hi - lo) * (i + 1) // n for i in range(n)]


def _lengths(c):
    """(cached lengths, drafted lengths) of a case's rows, before they are shuffled."""
    B, T, ctx = c["B"], c["T"], c["ctx"]
    return (_spread(B, ctx // 4, ctx) if c["ragged"] else [ctx] * B,
            _spread(B, (T + 1) // 2, T) if c["ragged"] else [T] * B)


def work(c):
    S, N = _lengths(c)
    B, T, H, D, e = c["B"], c["T"], c["kv_heads"], c["dim"], _size(c)
    if c["op"] == "append4":
        return {"bytes": 2 * c["layers"] * H * D * sum(N) * (2 + e), "flops": 0}
    if c["op"] == "evict":
        kept = [min(s, c["budget"]) for s in S]
        cut = sum(k for k, s in zip(kept, S) if k < s)
        return {"bytes": 2 * c["layers"] * H * D * cut * 2 * e + 4 * (sum(S) + sum(kept)), "flops": 0}
    toks, heads = sum(N), c["heads"]
    if c["op"] == "weights":
        return {"bytes": sum(S) * (H * D * e + 4 * (2 if c["decay"] else 1)) + toks * heads * (2 * D + 4),
                "flops": 2.0 * heads * D * sum(S) * toks / B}
    keys = sum(S) if c["op"] == "attn4" else sum(min(s, c["window"] + c["sinks"]) for s in S)
    io = 2 * (keys + toks) * H * D * e + toks * heads * (4 * D + 4)
    table = 4 * sum(-(-(k + n) // c["page"]) for k, n in zip(S if c["op"] == "attn4" else [keys // B] * B, N))
    return {"bytes": io + table, "flops": 4.0 * heads * D * (keys * toks / B + toks)}


# ----------------------------------------------------------------- inputs ---
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _shuffled(values, g):
    t = torch.tensor(values, dtype=torch.int32, device=DEV)
    return t[torch.randperm(len(values), generator=g, device=DEV)].contiguous()


def _rand(g, *shape):
    return torch.rand(shape, generator=g, device=DEV)


def _parents(g, B, T):
    """Random trees: parents drawn among the last nodes before, the root first."""
    i = torch.arange(T, device=DEV)
    back = 1 + (_rand(g, B, T) ** 2 * torch.clamp(i, max=12)).long()
    p = torch.clamp(i - back, min=0)
    p[:, 0] = -1
    return p.to(torch.int32)


def _power(byte):
    """2^(byte - 127), for bytes of 1 to 254."""
    return (byte.int() << 23).view(torch.float32)


def _quantise(x):
    """(codes, scale bytes) of values [..., dim] in the 4-bit format, two codes a byte."""
    b = x.reshape(*x.shape[:-1], -1, 32).float()
    m, k = torch.frexp(b.abs().amax(-1))
    e = torch.where(m == 0, -123, torch.where(m <= 0.875, k - 3, k - 2)).clamp(-123, 125)
    y = b.abs() * _power(127 - e)[..., None]
    step = torch.where(y < 2, 0.5, torch.where(y < 4, 1.0, 2.0))
    y = (torch.round(y / step) * step).clamp(max=6.0)
    code = torch.bucketize(y, torch.tensor(GRID, device=x.device)) + torch.where(b < 0, 8, 0)
    code = code.reshape(*x.shape[:-1], -1, 2).to(torch.uint8)
    return code[..., 0] | (code[..., 1] << 4), (e + 127).to(torch.uint8)


def _pairs():
    """[256, 2]: the two values of every byte."""
    grid = torch.tensor(GRID + tuple(-x for x in GRID), device=DEV)
    byte = torch.arange(256, device=DEV)
    return torch.stack([grid[byte & 15], grid[byte >> 4]], -1)


def _values4(pairs, codes, scales):
    """The values [..., dim] that codes and scale bytes stand for."""
    v = pairs[codes.int()].reshape(*scales.shape, 32)
    return (v * _power(scales)[..., None]).reshape(*codes.shape[:-1], -1)


def _cache(c, g, pool, scale):
    """A cache [layers, pages, slots, heads, dim] of normal values, and its 4-bit scales or None: layer by layer, as a
    model's layers fill it."""
    L, P, H, D = c.get("layers", 1), c["page"], c["kv_heads"], c["dim"]
    shape = (pool, H, P, D) if c["layout"] == "heads" else (pool, P, H, D)
    turn = (lambda t: t.transpose(2, 3)) if c["layout"] == "heads" else (lambda t: t)
    got = []
    for layer in range(L):
        x = torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16)
        if c["cache"] == "mxfp4":
            got.append(_quantise(x))
        elif c["cache"] == "e4m3":
            s = scale[layer][:, None] if c["layout"] == "tokens" else scale[layer][:, None, None]
            got.append(((x.float() / s).clamp(-448, 448).to(torch.float8_e4m3fn),))
        else:
            got.append((x,))
    whole = [torch.stack(t) if L > 1 else t[0][None] for t in zip(*got)]
    if c["cache"] == "mxfp4":
        return (turn(whole[0]).view(torch.float4_e2m1fn_x2), turn(whole[1]).view(torch.float8_e8m0fnu))
    return turn(whole[0]), scale


def prepare(c, seed):
    g = _gen(seed)
    B, T = c["B"], c["T"]
    S, N = _lengths(c)
    P, H, D, L = c["page"], c["kv_heads"], c["dim"], c.get("layers", 1)
    st = dict(case=c, T=T, B=B, pairs=_pairs())
    seq = _shuffled(S, g)
    if c["op"] == "evict":
        return _prepare_evict(c, st, g, seq)
    st["seq_len"] = seq
    st["block_len"] = _shuffled(N, g) if c["ragged"] else None
    cols = -(-(c["ctx"] + T) // P)
    pool = B * cols + 3
    st["table"] = torch.randperm(pool, generator=g, device=DEV)[:B * cols].view(B, cols).to(torch.int32).contiguous()
    scale = [0.01 + 0.02 * _rand(g, L, H) if c["cache"] == "e4m3" else None for _ in range(2)]
    st["k"], st["k_scale"] = _cache(c, g, pool, scale[0])
    if c["op"] != "weights":
        st["v"], st["v_scale"] = _cache(c, g, pool, scale[1])
    if c["op"] == "append4":
        for n in ("k_new", "v_new"):
            st[n] = torch.randn((L, B, T, H, D), generator=g, device=DEV, dtype=torch.bfloat16)
        # where the written rows are read back from
        pos = seq.long()[:, None] + torch.arange(T, device=DEV)
        st["at"] = st["table"].gather(1, pos // P).long(), pos % P
        st["live"] = _live(st["block_len"], B, T, DEV)[None, :, :, None, None]
        return st
    for n in ("k", "v", "k_scale", "v_scale"):  # these read one layer
        if st.get(n) is not None:
            st[n] = st[n][0]
    st["q"] = (2.5 * torch.randn((B, T, c["heads"], D), generator=g, device=DEV)).to(torch.bfloat16)
    if c["op"] == "weights":
        # what the attention before has left, and the sums so far
        st["lse"] = _plain_weights(st, lse_only=True)
        st["weights"] = torch.zeros((B, cols * P), device=DEV)
        st["was"] = torch.where(torch.arange(cols * P, device=DEV)[None, :] < seq[:, None], _rand(g, B, cols * P), 0.0)
        return st
    st["mask"] = st["depth"] = None
    if c.get("tree"):
        up = _ancestors(_parents(g, B, T))
        st["mask"] = _pack(up, T)
        st["depth"] = (up.sum(-1) - 1).to(torch.int32)
    st["out"] = torch.zeros_like(st["q"])
    st["lse"] = torch.zeros((B, T, c["heads"]), device=DEV)
    return st


def _prepare_evict(c, st, g, seq):
    """A pool whose rows hold their positions, with room for one copy of what they keep.  `now` is what a call
    updates in place, in one buffer; `was` is what it held before."""
    B, P, cols = c["B"], c["page"], -(-c["ctx"] // c["page"])
    held = (seq + P - 1) // P
    pool = B * cols + B * -(-c["budget"] // P) + 5
    ids = torch.randperm(pool, generator=g, device=DEV)[:B * cols].view(B, cols).to(torch.int32)
    have = torch.arange(cols, device=DEV)[None, :] < held[:, None]
    table = torch.where(have, ids, -1).to(torch.int32)
    count = torch.zeros(pool + 1, dtype=torch.int32, device=DEV)
    count[torch.where(have, ids, pool).view(-1).long()] = 1
    # sums of softmax weights: a few positions hold most of it, and many have next to none, or nothing
    w = torch.exp(2.5 * torch.randn((B, cols * P), generator=g, device=DEV)) * (_rand(g, B, cols * P) > 0.2)
    w = torch.where(torch.arange(cols * P, device=DEV)[None, :] < seq[:, None], w, 0.0)
    parts = [table.view(-1), held.to(torch.int32), seq, count[:pool], w.view(-1).view(torch.int32)]
    st["was"] = torch.cat(parts)
    st["now"] = st["was"].clone()
    t, st["row_pages"], st["seq_len"], st["refcount"], w = st["now"].split([p.numel() for p in parts])
    st["table"], st["weights"] = t.view(B, cols), w.view(torch.float32).view(B, cols * P)
    st["budget"] = torch.full((B,), c["budget"], dtype=torch.int32, device=DEV)
    st["k"], _ = _cache(c, g, pool, None)
    st["v"], _ = _cache(c, g, pool, None)
    return st


# ------------------------------------------------------------- plain forms ---
def _ancestors(parent):
    """[B, T, T] truth values: node j is i or above i.  (I + M)^T counts walks along the parent links M; the counts
    are below 2^256, which 64 bits hold, and none is lost to rounding since all are sums of positives."""
    B, T = parent.shape
    j = torch.arange(T, device=parent.device)
    link = (parent[:, :, None] == j) | (j[:, None] == j[None, :])
    return torch.matrix_power(link.double(), T) > 0


def _pack(vis, T):
    """Truth values [B, T, T] as bits, 32 to a word."""
    B, words = vis.shape[0], (T + 31) // 32
    full = torch.zeros((B, T, words * 32), dtype=torch.int64, device=vis.device)
    full[:, :, :T] = vis
    w = (full.view(B, T, words, 32) << torch.arange(32, device=vis.device)).sum(-1)
    return torch.where(w >= 2 ** 31, w - 2 ** 32, w).to(torch.int32)


def _live(block_len, B, T, device):
    t = torch.arange(T, device=device)
    return (t[None, :] < block_len[:, None]) if block_len is not None else torch.ones((B, T), dtype=torch.bool, device=device)


def _rows(x, table, pos):
    """Rows [B, n, heads, ...] of a cache [pages, slots, heads, ...] at positions [B, n]."""
    P = x.shape[1]
    page = table.gather(1, (pos // P).clamp(max=table.shape[1] - 1)).long()
    return x[page, pos % P]


def _read(s, name, pos):
    """Rows [B, n, heads, dim] of K or V as the 32-bit values that they stand for."""
    x, scale, table = s[name], s[name + "_scale"], s["table"]
    if x.dtype is torch.float4_e2m1fn_x2:
        return _values4(s["pairs"], _rows(x.view(torch.uint8), table, pos), _rows(scale.view(torch.uint8), table, pos))
    r = _rows(x.view(torch.uint8), table, pos).view(x.dtype) if x.dtype is torch.float8_e4m3fn else _rows(x, table, pos)
    return r.float() * scale[:, None] if scale is not None else r.float()


def _scores(q, K):
    """[B, heads, T * group, n] scores of every query and key."""
    B, T, Hq, D = q.shape
    H = K.shape[2]
    Q = q.float().view(B, T, H, Hq // H, D).permute(0, 2, 1, 3, 4).reshape(B, H, T * (Hq // H), D)
    return torch.matmul(Q, K.permute(0, 2, 3, 1).contiguous()) * D ** -0.5


def _seen_nodes(s, node):
    """[B, T, n]: what the mask says of the drafted nodes at these places (a chain's: those up to itself)."""
    T = s["T"]
    at = node.clamp(0, T - 1).long()
    if s["mask"] is None:
        return at[:, None, :] <= torch.arange(T, device=DEV)[None, :, None]
    word = torch.gather(s["mask"], 2, (at >> 5)[:, None, :].expand(-1, T, -1))
    return (word >> (at & 31)[:, None, :]) & 1 == 1


def _softmax(s, z, vis, V):
    """(out, lse) of scores [B, heads, T * group, n] under truth values [B, T, n]."""
    B, T, Hq, D = s["q"].shape
    H = V.shape[2]
    n = z.shape[-1]
    z = z.view(B, H, T, Hq // H, n).masked_fill(~vis[:, None, :, None, :], -math.inf)
    top = z.amax(-1, keepdim=True).clamp(min=-3e38)
    p = torch.exp(z - top)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(B, H, -1, n), V.permute(0, 2, 1, 3).contiguous()).view(B, H, T, Hq // H, D)
    o = torch.where(total > 0, o / total, 0.0)
    lse = (top + torch.log(total)).squeeze(-1).permute(0, 2, 1, 3).reshape(B, T, Hq)
    o = o.permute(0, 2, 1, 3, 4).reshape(B, T, Hq, D)
    live = _live(s["block_len"], B, T, DEV)
    return (torch.where(live[:, :, None, None], o, 0.0).to(torch.bfloat16),
            torch.where(live[:, :, None], lse, 0.0))


def _plain_attn4(s):
    B, T = s["B"], s["T"]
    n = s["table"].shape[1] * s["case"]["page"]
    pos = torch.arange(n, device=DEV)[None, :].expand(B, n)
    node = pos - s["seq_len"][:, None]
    inside = node < _live(s["block_len"], B, T, DEV).sum(1, keepdim=True)
    K, V = (_read(s, x, pos) for x in "kv")
    vis = (_seen_nodes(s, node) | (node < 0)[:, None, :]) & inside[:, None, :]
    return _softmax(s, _scores(s["q"], K), vis, V)


def _plain_window(s):
    """Only the positions that some query may see are read: the sinks, and the window before the tokens."""
    c, B, T = s["case"], s["B"], s["T"]
    W, A = c["window"], c["sinks"]
    seq = s["seq_len"].long()[:, None]
    behind = (seq - W + 1).clamp(min=A) + torch.arange(min(W, c["ctx"]) + T, device=DEV)
    first = torch.arange(min(A, c["ctx"] + T), device=DEV)[None, :].expand(B, -1)
    pos = torch.cat([first, behind], 1)
    node = pos - seq
    inside = node < _live(s["block_len"], B, T, DEV).sum(1, keepdim=True)
    depth = s["depth"].long() if s["depth"] is not None else torch.arange(T, device=DEV)[None, :].expand(B, T)
    key = torch.where(node < 0, pos, seq + depth.gather(1, node.clamp(0, T - 1)))
    near = (key < A)[:, None, :] | ((seq + depth)[:, :, None] - key[:, None, :] < W)
    vis = (_seen_nodes(s, node) | (node < 0)[:, None, :]) & inside[:, None, :] & near
    K, V = (_read(s, x, pos) for x in "kv")
    return _softmax(s, _scores(s["q"], K), vis, V)


def _plain_weights(s, lse_only=False):
    c, B, T = s["case"], s["B"], s["T"]
    n = s["table"].shape[1] * c["page"]
    pos = torch.arange(n, device=DEV)[None, :].expand(B, n)
    cached = pos < s["seq_len"][:, None]
    z = _scores(s["q"], _read(s, "k", pos)).view(B, c["kv_heads"], T, -1, n)
    z = z.masked_fill(~cached[:, None, None, None, :], -math.inf)
    if lse_only:  # the tokens themselves, which the attention saw too, weigh as one more key of score 0
        return torch.logaddexp(z.logsumexp(-1), torch.zeros((), device=DEV)).permute(0, 2, 1, 3).reshape(B, T, -1).contiguous()
    lse = s["lse"].view(B, T, c["kv_heads"], -1).permute(0, 2, 1, 3)
    live = _live(s["block_len"], B, T, DEV)
    p = torch.where(live[:, None, :, None, None], torch.exp(z - lse[..., None]), 0.0)
    return torch.where(cached, c["decay"] * s["weights"] + p.sum((1, 2, 3)), s["weights"])


def _plain_append4(s):
    c = s["case"]
    L, B, T, H, D, P = c["layers"], s["B"], s["T"], c["kv_heads"], c["dim"], c["page"]
    pos = s["seq_len"].long()[:, None] + torch.arange(T, device=DEV)
    live = _live(s["block_len"], B, T, DEV).view(-1).nonzero().view(-1)
    page = s["table"].gather(1, pos // P).long().view(-1)[live]
    slot = (pos % P).view(-1)[live]

    def write(x, scale, new):
        code, byte = _quantise(new.view(L, B * T, H, D)[:, live])
        x.view(torch.uint8)[:, page, slot] = code
        scale.view(torch.uint8)[:, page, slot] = byte

    write(s["k"], s["k_scale"], s["k_new"])
    write(s["v"], s["v_scale"], s["v_new"])
    return _written(s)


def _written(s):
    """The values that the rows of the new tokens now hold: [layers, B, T, heads, dim], zeros past a row's tokens."""
    page, slot = s["at"]
    return tuple(torch.where(s["live"], _values4(s["pairs"], s[n].view(torch.uint8)[:, page, slot],
                                                 s[n + "_scale"].view(torch.uint8)[:, page, slot]), 0.0) for n in "kv")


def _plain_evict(s):
    c, B = s["case"], s["B"]
    P, cols, K = c["page"], s["table"].shape[1], c["budget"]
    pos = torch.arange(cols * P, device=DEV)[None, :]
    n = s["seq_len"].long()[:, None]
    cut = n > s["budget"][:, None]
    stays = (pos < c["sinks"]) | (pos >= n - c["recent"])
    value = torch.where(pos < n, torch.where(stays, math.inf, s["weights"]), -1.0)
    order = torch.sort(value, dim=1, descending=True, stable=True).indices[:, :K]
    kept = torch.sort(order, dim=1).values
    # the lowest free pages, in row order
    need = torch.where(cut, -(-K // P), 0).view(-1)
    free = s["refcount"] == 0
    granted = need.sum() <= free.sum()
    need = torch.where(granted, need, 0)
    cut = cut & granted
    ids = torch.sort((~free).to(torch.int8), stable=True).indices
    start = need.cumsum(0) - need
    col = torch.arange(cols, device=DEV)[None, :]
    fresh = ids[(start[:, None] + col).clamp(max=ids.numel() - 1)].to(torch.int32)
    take = col < need[:, None]
    # the kept rows into them
    row = cut.expand(B, kept.shape[1]).reshape(-1).nonzero().view(-1)
    to = torch.arange(kept.shape[1], device=DEV)[None, :].expand(B, -1)
    place = lambda t, p: (t.gather(1, p // P).long() * P + p % P).view(-1)[row]  # noqa: E731
    come, go = place(s["table"], kept), place(fresh, to)
    for x in (s["k"], s["v"]):
        flat = x.view(x.shape[0], -1, *x.shape[3:])
        flat[:, go] = flat[:, come]
    # the pool, the table and the weights
    held = (col < s["row_pages"][:, None]) & cut
    one = torch.ones_like(s["table"])
    s["refcount"].index_add_(0, torch.where(held, s["table"], 0).view(-1).long(), torch.where(held, -one, 0).view(-1))
    s["refcount"].index_add_(0, torch.where(take, fresh, 0).view(-1).long(), torch.where(take, one, 0).view(-1))
    s["table"].copy_(torch.where(cut, torch.where(take, fresh, -1), s["table"]))
    moved = torch.zeros_like(s["weights"])
    moved[:, :kept.shape[1]] = s["weights"].gather(1, kept)
    s["weights"].copy_(torch.where(cut, moved, s["weights"]))
    s["row_pages"].copy_(torch.where(cut.view(-1), -(-K // P), s["row_pages"]))
    s["seq_len"].copy_(torch.where(cut.view(-1), K, s["seq_len"]))
    return _evicted(s, granted.to(torch.int32).view(1))


def _evicted(s, granted):
    return s["k"], s["v"], s["table"], s["row_pages"], s["seq_len"], s["refcount"], s["weights"], granted


# ------------------------------------------------------------------- passes ---
def run(s):
    op = s["case"]["op"]
    if op == "evict":
        s["now"].copy_(s["was"])
    if op == "weights" and s["case"]["decay"]:
        s["weights"].copy_(s["was"])
    if own:
        return _library(s, op)
    return {"attn4": _plain_attn4, "append4": _plain_append4, "window": _plain_window, "weights": _plain_weights,
            "evict": _plain_evict}[op](s)


def _library(s, op):
    import draft_selection_amd as ds

    c = s["case"]
    if op == "evict":
        pages = ds.Pages(s["table"], s["row_pages"], s["seq_len"], s["refcount"], c["page"])
        return _evicted(s, ds.cache_evict(pages, s["budget"], s["weights"], s["k"], s["v"], sinks=c["sinks"],
                                          recent=c["recent"]))
    if op == "append4":
        ds.cache_append(s["k_new"], s["v_new"], s["k"], s["v"], s["table"], s["seq_len"], block_len=s["block_len"],
                        k_scale=s["k_scale"], v_scale=s["v_scale"])
        return _written(s)
    if op == "weights":
        return ds.key_weights(s["q"], s["lse"], s["k"], s["table"], s["seq_len"], s["weights"], block_len=s["block_len"],
                              decay=c["decay"], k_scale=s["k_scale"])
    kw = dict(mask=s["mask"], block_len=s["block_len"], k_scale=s["k_scale"], v_scale=s["v_scale"], out=s["out"], lse=s["lse"])
    if op == "attn4":
        return ds.tree_attn(s["q"], s["k"], s["v"], s["table"], s["seq_len"], **kw)
    return ds.tree_attn_window(s["q"], s["k"], s["v"], s["table"], s["seq_len"], c["window"], sinks=c["sinks"],
                               depth=s["depth"], **kw)


# ------------------------------------------------------------------- exact ---
def exact(c, seed):
    """The definition in 64 bits, sequence by sequence.  Outputs that are whole numbers, or copies of inputs, have none."""
    if c["op"] == "evict":
        return None
    s = prepare(c, seed)
    D, P, T = c["dim"], c["page"], c["T"]
    lengths = s["block_len"].tolist() if s["block_len"] is not None else [T] * c["B"]

    def held(name, pages, n):
        """The first n positions of these pages, [n, heads, dim]."""
        x = s[name]
        if c["cache"] == "mxfp4":
            byte = x.view(torch.uint8)[pages]
            code = torch.stack([byte & 15, byte >> 4], -1).flatten(-2).int()
            low, up = code & 1, (code >> 1) & 3  # one bit behind the leading one, two of exponent
            size = torch.where(up == 0, 0.5 * low.double(), (1 + 0.5 * low) * torch.exp2(up.double() - 1))
            x = torch.where(code >= 8, -size, size)
            power = torch.exp2(s[name + "_scale"].view(torch.uint8)[pages].double() - 127)
            x = x * power.repeat_interleave(32, -1)
        else:
            x = x[pages].to(torch.float64)
            if c["cache"] == "e4m3":
                x = x * s[name + "_scale"].double()[:, None]
        return x.reshape(-1, *x.shape[2:])[:n]

    def grid4(x):
        """The nearest values of the 4-bit format, by the distance to each."""
        b = x.to(torch.float64).reshape(*x.shape[:-1], -1, 32)
        e = torch.ceil(torch.log2(b.abs().amax(-1, keepdim=True) / 7)).clamp(-123, 125)
        y = b / torch.exp2(e)
        grid = torch.tensor(GRID, dtype=torch.float64, device=DEV)
        best = torch.zeros_like(y)
        gap = torch.full_like(y, math.inf)
        for i in (0, 2, 4, 6, 1, 3, 5, 7):  # even codes first: they win ties
            d = (y.abs() - grid[i]).abs()
            best, gap = torch.where(d < gap, grid[i], best), torch.minimum(d, gap)
        return (torch.copysign(best, y) * torch.exp2(e)).reshape(x.shape)

    if c["op"] == "append4":
        out = [torch.zeros(s["k_new"].shape, dtype=torch.float64, device=DEV) for _ in range(2)]
        for o, new in zip(out, (s["k_new"], s["v_new"])):
            for b, n in enumerate(lengths):
                o[:, b, :n] = grid4(new[:, b, :n])
        return tuple(out)
    H, Hq = c["kv_heads"], c["heads"]
    group = Hq // H
    if c["op"] == "weights":
        got = (s["was"] if c["decay"] else s["weights"]).double()
        for b, n in enumerate(lengths):
            done = int(s["seq_len"][b])
            K = held("k", s["table"][b, :(done + P - 1) // P].long(), done)
            total = torch.zeros(done, dtype=torch.float64, device=DEV)
            for h in range(Hq):
                z = torch.mm(s["q"][b, :n, h].double(), K[:, h // group].T.contiguous()) / math.sqrt(D)
                total += torch.exp(z - s["lse"][b, :n, h].double()[:, None]).sum(0)
            got[b, :done] = c["decay"] * got[b, :done] + total
        return got
    out = torch.zeros((c["B"], T, Hq, D), dtype=torch.float64, device=DEV)
    lse = torch.zeros((c["B"], T, Hq), dtype=torch.float64, device=DEV)
    for b, n in enumerate(lengths):
        done = int(s["seq_len"][b])
        pages = s["table"][b, :(done + n + P - 1) // P].long()
        words = s["mask"][b, :n].cpu().tolist() if s["mask"] is not None else None
        sees = torch.ones((n, done + n), dtype=torch.bool)
        sees[:, done:] = torch.tensor([[j <= i if words is None else (words[i][j // 32] >> (j % 32)) & 1 == 1 for j in range(n)]
                                       for i in range(n)])
        if c["op"] == "window":
            deep = s["depth"][b, :n].cpu().long() if s["depth"] is not None else torch.arange(n)
            at = torch.cat([torch.arange(done), done + deep])
            sees &= (at < c["sinks"])[None, :] | (at[None, :] > (done + deep)[:, None] - c["window"])
        some = sees.any(0).nonzero().view(-1)
        bias = torch.zeros((n, len(some)), dtype=torch.float64)
        bias[~sees[:, some]] = -math.inf
        bias, some = bias.to(DEV), some.to(DEV)
        K, V = (held(x, pages, done + n)[some] for x in "kv")
        for h in range(Hq):
            z = torch.mm(s["q"][b, :n, h].double(), K[:, h // group].T.contiguous()) / math.sqrt(D) + bias
            lse[b, :n, h] = torch.logsumexp(z, dim=1)
            out[b, :n, h] = torch.mm(torch.softmax(z, dim=1), V[:, h // group].contiguous())
    return out, lse
