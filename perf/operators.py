"""The cache side of verifying drafted tokens, as it is measured.

Four operators, each in its plain form (elementary torch operations) and as the library's calls:

  attn    attention of a tree of drafted tokens over a paged K/V cache (tree_attn)
  tree    a tree's ancestor mask and depths, and the path of it that the target keeps (tree_mask, tree_accept)
  cache   one step's writes: the drafted tokens' rows appended, the kept ones moved together (cache_append,
          cache_compact)
  pages   one step of the page pool: losing rows freed, their parents forked into them, pages reserved for the
          next block (pages_free, pages_fork, pages_reserve)

Every pass leaves a state from which the same pass gives the same outputs.
"""
import math

import torch

own = False
DEV = "cuda"


# ------------------------------------------------------------------ cases ---
def _attn(name, B, T, ctx, heads, kv_heads, dim, page, cache="bf16", tree=True, ragged=True):
    c = dict(op="attn", B=B, T=T, ctx=ctx, heads=heads, kv_heads=kv_heads, dim=dim, page=page, cache=cache, tree=tree,
             ragged=ragged)
    return dict(c, name=name) if name else c


def _tree(name, B, T, ragged=True):
    c = dict(op="tree", B=B, T=T, ragged=ragged)
    return dict(c, name=name) if name else c


def _cache(name, B, T, ctx, layers, kv_heads, dim, page, cache="bf16", ragged=True):
    c = dict(op="cache", B=B, T=T, ctx=ctx, layers=layers, kv_heads=kv_heads, dim=dim, page=page, cache=cache,
             ragged=ragged)
    return dict(c, name=name) if name else c


def _pages(name, rows, forks, ctx, layers, kv_heads, dim, page, T):
    c = dict(op="pages", B=rows, forks=forks, ctx=ctx, layers=layers, kv_heads=kv_heads, dim=dim, page=page, T=T)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one sequence, one token, a short cache: plain decoding between drafts, where latency counts
        _attn("attn_one_token", 1, 1, 333, 32, 8, 128, 16, tree=False, ragged=False),
        # small drafted blocks (8 and the verified token) as chains, ragged, at 27B-class blocks
        _attn("attn_chain9", 32, 9, 2048, 32, 8, 128, 16, tree=False),
        # the batched throughput shape: 64 blocks of 16 and the verified token, as chains
        _attn("attn_chain17", 64, 17, 4096, 32, 8, 128, 32, tree=False),
        # trees of 64 nodes over long caches: more arithmetic than bytes
        _attn("attn_tree64", 8, 64, 16384, 32, 8, 128, 64),
        # two very long sequences with an 8-bit cache, trees of 32
        _attn("attn_long_e4m3", 2, 32, 131000, 32, 8, 128, 64, cache="e4m3", ragged=False),
        # wide heads, few of them
        _attn("attn_tree21_wide", 16, 21, 5000, 16, 2, 256, 16),
        # one tree after its target pass, and a large batch of the longest trees
        _tree("tree_one", 1, 60, ragged=False),
        _tree("tree_batch", 256, 256),
        # one layer's write of an 8-bit cache at a small batch, and every layer of the batched shape
        _cache("cache_layer_e4m3", 8, 9, 500, 1, 8, 128, 16, cache="e4m3"),
        _cache("cache_layers", 64, 17, 200, 36, 8, 128, 16),
        # a few rows of a small pool, and a large table with 48 forks over eight layers
        _pages("pages_small", 8, 4, 700, 1, 8, 128, 16, 9),
        _pages("pages_layers", 128, 48, 600, 8, 8, 128, 64, 17),
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
        op = rng.choice(["attn", "attn", "attn", "tree", "cache", "pages"])
        if op == "attn":
            kv = rng.choice([1, 2, 4, 8])
            tree = rng.random() < 0.6
            c = _attn(None, _span(rng, 1, 64), _span(rng, 1, 100 if tree else 33), _span(rng, 1, 60000),
                      kv * rng.choice([1, 2, 4, 5, 8]), kv, rng.choice([64, 80, 128, 128, 128, 256]),
                      rng.choice([8, 16, 32, 48, 64, 128]), rng.choice(["bf16", "bf16", "e4m3"]), tree,
                      rng.random() < 0.7)
        elif op == "tree":
            c = _tree(None, _span(rng, 1, 256), _span(rng, 1, 256), rng.random() < 0.7)
        elif op == "cache":
            c = _cache(None, _span(rng, 1, 64), _span(rng, 1, 64), _span(rng, 1, 800), _span(rng, 1, 36),
                       rng.choice([1, 2, 4, 8]), rng.choice([64, 80, 128, 256]), rng.choice([8, 16, 32, 48, 64]),
                       rng.choice(["bf16", "bf16", "e4m3"]), rng.random() < 0.7)
        else:
            rows = _span(rng, 2, 256)
            c = _pages(None, rows, max(1, rows // rng.choice([2, 3, 4, 8])), _span(rng, 1, 1000), _span(rng, 1, 36),
                       rng.choice([1, 2, 4, 8]), rng.choice([64, 80, 128, 256]), rng.choice([8, 16, 32, 48, 64]),
                       _span(rng, 1, 64))
        w = work(c)
        if all(w[k] <= top[op, k] for k in w) and _held(c) < 4e9:
            return c


def _held(c):
    """Bytes of the caches (both operands) that a case holds."""
    e = 1 if c.get("cache") == "e4m3" else 2
    if c["op"] == "tree":
        return 0
    return 2 * c.get("layers", 1) * c["B"] * (c["ctx"] + c["T"] + c["page"]) * c["kv_heads"] * c["dim"] * e


def _spread(n, lo, hi):
    """n lengths from lo to hi, evenly."""
    return [lo + (hi - lo) * (i + 1) // n for i in range(n)]


def _lengths(c):
    """(cached lengths, drafted lengths) of a case's rows, before they are shuffled."""
    B, T = c["B"], c["T"]
    ragged = c.get("ragged", True)
    ctx = c.get("ctx", 0)
    return (_spread(B, ctx // 4, ctx) if ragged else [ctx] * B,
            _spread(B, (T + 1) // 2, T) if ragged and c["op"] != "pages" else [T] * B)


def _kept(n):
    """Nodes of a path that a tree of n may keep, on average, in the cases here."""
    return 1 + (n - 1) // 4


def work(c):
    S, N = _lengths(c)
    B, T = c["B"], c["T"]
    if c["op"] == "attn":
        e = 1 if c["cache"] == "e4m3" else 2
        keys, toks = sum(S), sum(N)
        io = 2 * (keys + toks) * c["kv_heads"] * c["dim"] * e + toks * c["heads"] * (4 * c["dim"] + 4)
        pairs = keys * toks / B + toks
        table = 4 * sum(-(-(s + n) // c["page"]) for s, n in zip(S, N))
        return {"bytes": io + table, "flops": 4.0 * c["heads"] * c["dim"] * pairs}
    if c["op"] == "tree":
        words = (T + 31) // 32
        return {"bytes": sum(N) * (4 + 4 * words + 4 + 12) + 8 * B * T, "flops": 0}
    row = c.get("layers", 1) * 2 * c["kv_heads"] * c["dim"]
    if c["op"] == "cache":
        e = 1 if c["cache"] == "e4m3" else 2
        return {"bytes": row * (sum(N) * (2 + e) + sum(_kept(n) - 1 for n in N) * 2 * e), "flops": 0}
    part = sum(s % c["page"] for s in S) * c["forks"] / B
    held = sum(-(-s // c["page"]) for s in S) * c["forks"] / B
    return {"bytes": part * row * 2 * 2 + held * 4 * 6, "flops": 0}


# ----------------------------------------------------------------- inputs ---
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _shuffled(values, g):
    t = torch.tensor(values, dtype=torch.int32, device=DEV)
    return t[torch.randperm(len(values), generator=g, device=DEV)].contiguous()


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV)


def _rand(g, *shape):
    return torch.rand(shape, generator=g, device=DEV)


def _parents(g, B, T):
    """Random trees: parents drawn among the last nodes before, the root first."""
    i = torch.arange(T, device=DEV)
    back = 1 + (_rand(g, B, T) ** 2 * torch.clamp(i, max=12)).long()
    p = torch.clamp(i - back, min=0)
    p[:, 0] = -1
    return p.to(torch.int32)


def _values(g, scale, *shape):
    """Cached values [layers, pages, slots, heads, dim]: normal ones, in e4m3 over a scale for each layer and head."""
    x = torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16)
    return x if scale is None else (x.float() / scale[:, None, None, :, None]).clamp(-448, 448).to(torch.float8_e4m3fn)


def _tokens(g, parent, vocab=151936):
    """Drafted tokens, and the target's token after each node: that of one of its children mostly.  As the
    library's top-16 lists give it, the target's choice is the first of 16 ids."""
    B, T = parent.shape
    tok = torch.randint(vocab, (B, T), generator=g, device=DEV, dtype=torch.int32)
    top = torch.randint(vocab, (B, T, 16), generator=g, device=DEV, dtype=torch.int32)
    # the last node that names a parent (in a shuffled order) is the child its target agrees with
    score = _rand(g, B, T)
    child = (parent[:, None, :] == torch.arange(T, device=DEV)[None, :, None]) * (0.5 + score[:, None, :])
    best, which = child.max(dim=2)
    agree = (best > 0) & (_rand(g, B, T) < 0.9)
    top[:, :, 0] = torch.where(agree, tok.gather(1, which), top[:, :, 0])
    return tok, top


def prepare(c, seed):
    g = _gen(seed)
    B, T = c["B"], c["T"]
    S, N = _lengths(c)
    st = dict(case=c, T=T, B=B)
    if c["op"] == "tree":
        st["parent"] = _parents(g, B, T)
        st["block_len"] = _shuffled(N, g) if c["ragged"] else None
        st["tok"], st["top"] = _tokens(g, st["parent"])
        st["mask"] = torch.zeros((B, T, (T + 31) // 32), dtype=torch.int32, device=DEV)
        st["depth"] = torch.zeros((B, T), dtype=torch.int32, device=DEV)
        return st
    P, H, D, L = c["page"], c["kv_heads"], c["dim"], c.get("layers", 1)
    seq = _shuffled(S, g)
    st["seq_len"] = seq
    cols = -(-(c["ctx"] + T) // P)
    e4m3 = c.get("cache") == "e4m3"
    if c["op"] == "pages":
        return _prepare_pages(c, st, g, cols)
    st["block_len"] = _shuffled(N, g) if c["ragged"] else None
    pool = B * cols + 3
    st["table"] = torch.randperm(pool, generator=g, device=DEV)[:B * cols].view(B, cols).to(torch.int32).contiguous()
    if e4m3:
        st["k_scale"] = 0.01 + 0.02 * _rand(g, L, H)
        st["v_scale"] = 0.01 + 0.02 * _rand(g, L, H)
    st["k"] = _values(g, st.get("k_scale"), L, pool, P, H, D)
    st["v"] = _values(g, st.get("v_scale"), L, pool, P, H, D)
    if c["op"] == "attn":
        st["k"], st["v"] = st["k"][0], st["v"][0]
        st["q"] = (2.5 * _randn(g, B, T, c["heads"], D)).to(torch.bfloat16)
        st["mask"] = _pack(_ancestors(_parents(g, B, T)), T) if c["tree"] else None
        st["out"] = torch.zeros_like(st["q"])
        st["lse"] = torch.zeros((B, T, c["heads"]), device=DEV)
        return st
    # cache: one step's new rows, and the path that the target keeps of them
    st["k_new"] = _randn(g, L, B, T, H, D).to(torch.bfloat16)
    st["v_new"] = _randn(g, L, B, T, H, D).to(torch.bfloat16)
    parent = _parents(g, B, T)
    tok, top = _tokens(g, parent)
    st["n_keep"], st["path"], _ = _plain_accept(parent, tok, top[:, :, 0], st["block_len"])
    return st


def _prepare_pages(c, st, g, cols):
    """A pool in the middle of its work: the first rows are parents, the next `forks` ones hold what a branch left."""
    B, P, H, D, L, F = c["B"], c["page"], c["kv_heads"], c["dim"], c["layers"], c["forks"]
    keep = B - F
    row = torch.randperm(B, generator=g, device=DEV)
    child = row[:F]
    held = (st["seq_len"] + P - 1) // P
    pool = B * cols + 7
    ids = torch.randperm(pool, generator=g, device=DEV)[:B * cols].view(B, cols).to(torch.int32)
    have = torch.arange(cols, device=DEV)[None, :] < held[:, None]
    st["table"] = torch.where(have, ids, -1).to(torch.int32).contiguous()
    st["row_pages"] = held.to(torch.int32).contiguous()
    st["refcount"] = torch.zeros(pool + 1, dtype=torch.int32, device=DEV).index_add_(
        0, torch.where(have, ids, pool).view(-1).long(), torch.ones(B * cols, dtype=torch.int32, device=DEV))[:pool].clone()
    st["which"] = torch.zeros(B, dtype=torch.int32, device=DEV)
    st["which"][child] = 1
    st["src"] = torch.full((B,), -1, dtype=torch.int32, device=DEV)
    st["src"][child] = row[F + torch.randint(max(keep, 1), (F,), generator=g, device=DEV)].to(torch.int32) if keep else -1
    st["extra"] = torch.full((B,), c["T"], dtype=torch.int32, device=DEV)
    st["k"] = _values(g, None, L, pool, P, H, D)
    st["v"] = _values(g, None, L, pool, P, H, D)
    return st


# ------------------------------------------------------------- plain forms ---
def _ancestors(parent):
    """[B, T, T] truth values: node j is i or above i.  (I + M)^T' counts walks along the parent links M; they are
    below 2^256 for 256 nodes, which 64 bits hold, and none is lost to rounding since all are sums of positives."""
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


def _plain_attn(q, k, v, table, seq_len, mask, block_len, k_scale, v_scale):
    B, T, Hq, D = q.shape
    P, H = k.shape[1], k.shape[2]
    n = table.shape[1] * P
    live = _live(block_len, B, T, q.device)
    pos = torch.arange(n, device=q.device)
    node = pos[None, :] - seq_len[:, None]  # [B, n]: the drafted node at a position, negative before them
    inside = node < live.sum(1, keepdim=True)
    at = node.clamp(0, T - 1).long()
    if mask is None:
        seen = at[:, None, :] <= torch.arange(T, device=q.device)[None, :, None]
    else:
        word = torch.gather(mask, 2, (at >> 5)[:, None, :].expand(B, T, n))
        seen = (word >> (at & 31)[:, None, :]) & 1 == 1
    vis = (seen | (node < 0)[:, None, :]) & inside[:, None, :]
    K = k[table.long()].view(B, n, H, D).float()
    V = v[table.long()].view(B, n, H, D).float()
    if k_scale is not None:
        K, V = K * k_scale[:, None], V * v_scale[:, None]
    V = torch.where(inside[:, :, None, None], V, 0.0)
    Q = q.float().view(B, T, H, Hq // H, D).permute(0, 2, 1, 3, 4).reshape(B, H, T * (Hq // H), D)
    z = torch.matmul(Q, K.permute(0, 2, 3, 1).contiguous()) * D ** -0.5
    z = z.view(B, H, T, Hq // H, n).masked_fill(~vis[:, None, :, None, :], -math.inf)
    top = z.amax(-1, keepdim=True).clamp(min=-3e38)
    p = torch.exp(z - top)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(B, H, -1, n), V.permute(0, 2, 1, 3).contiguous()).view(B, H, T, Hq // H, D)
    o = torch.where(total > 0, o / total, 0.0)
    lse = (top + torch.log(total)).squeeze(-1).permute(0, 2, 1, 3).reshape(B, T, Hq)
    o = o.permute(0, 2, 1, 3, 4).reshape(B, T, Hq, D)
    return (torch.where(live[:, :, None, None], o, 0.0).to(torch.bfloat16),
            torch.where(live[:, :, None], lse, 0.0))


def _plain_mask(parent, block_len):
    B, T = parent.shape
    live = _live(block_len, B, T, parent.device)
    up = _ancestors(parent)
    return (torch.where(live[:, :, None], _pack(up, T), 0),
            torch.where(live, up.sum(-1) - 1, 0).to(torch.int32))


def _plain_accept(parent, tok, target, block_len):
    """A node is kept if it and everything above it is the lowest sibling with the token its parent's target wants."""
    B, T = parent.shape
    live = _live(block_len, B, T, parent.device)
    i = torch.arange(T, device=parent.device)
    up = parent.clamp(min=0).long()
    fits = (tok == target.gather(1, up)) & live & (i > 0)
    first = torch.full((B, T), T, device=parent.device).scatter_reduce(1, up, torch.where(fits, i, T), "amin")
    fits = (fits & (first.gather(1, up) == i)) | ((i == 0) & live)
    kept = ((_ancestors(parent) & ~fits[:, None, :]).sum(-1) == 0) & live
    n_keep = kept.sum(1)
    order = torch.where(kept, i, T).sort(dim=1).values
    path = torch.where(order < T, order, -1)
    want = target.gather(1, path.clamp(min=0))
    return (n_keep.to(torch.int32), path.to(torch.int32), torch.where(path >= 0, want, -1).to(torch.int32))


def _places(table, pos, P):
    """Flat row numbers (page * P + slot) of positions [B, n]."""
    return table.gather(1, (pos // P).clamp(max=table.shape[1] - 1)).long() * P + pos % P


def _plain_cache(s):
    c = s["case"]
    P, B, T = c["page"], s["B"], s["T"]
    L, H, D = c["layers"], c["kv_heads"], c["dim"]
    t = torch.arange(T, device=DEV)
    seq = s["seq_len"].long()[:, None]
    rows = _places(s["table"], seq + t, P)
    live = _live(s["block_len"], B, T, rows.device)
    i = live.view(-1).nonzero().view(-1)
    moved = (t[None, :] < s["n_keep"][:, None]).view(-1).nonzero().view(-1)
    come = _places(s["table"], seq + s["path"].clamp(min=0), P)

    def step(cache, new, scale):
        flat = cache.view(L, -1, H, D)
        x = new.view(L, B * T, H, D)[:, i]
        if scale is not None:
            x = (x.float() / scale[:, None, :, None]).clamp(-448, 448).to(cache.dtype)
            flat = flat.view(torch.uint8)
            x = x.view(torch.uint8)
        flat[:, rows.view(-1)[i]] = x
        flat[:, rows.view(-1)[moved]] = flat[:, come.view(-1)[moved]]
        return cache.float() if scale is not None else cache

    return (step(s["k"], s["k_new"], s.get("k_scale")), step(s["v"], s["v_new"], s.get("v_scale")),
            s["seq_len"] + s["n_keep"])


def _add_at(x, index, keep, value):
    """x[index] += value where keep holds."""
    x.index_add_(0, torch.where(keep, index, 0).view(-1).long(), (keep * value).view(-1).to(x.dtype))


def _give(s, need):
    """The lowest free pages to the rows that need some, in row order: (page, row) lists, or none if they do not suffice."""
    free = s["refcount"] == 0
    total = need.sum()
    need = torch.where(total <= free.sum(), need, 0)
    ids = torch.sort((~free).to(torch.int8), stable=True).indices
    start = need.cumsum(0) - need
    col = torch.arange(s["table"].shape[1], device=DEV)[None, :]
    take = col < need[:, None]
    page = ids[(start[:, None] + col).clamp(max=ids.numel() - 1)]
    _add_at(s["refcount"], page, take, 1)
    return need, take, page, total <= free.sum()


def _plain_pages(s):
    c = s["case"]
    P, L, H, D = c["page"], c["layers"], c["kv_heads"], c["dim"]
    table, cols = s["table"], torch.arange(s["table"].shape[1], device=DEV)[None, :]
    # free
    gone = s["which"] != 0
    _add_at(s["refcount"], table, (cols < s["row_pages"][:, None]) & gone[:, None], -1)
    table.masked_fill_(gone[:, None], -1)
    s["row_pages"].masked_fill_(gone, 0)
    s["seq_len"].masked_fill_(gone, 0)
    # fork
    at = s["src"].clamp(min=0).long()
    child = s["src"] >= 0
    size = torch.where(child, s["seq_len"][at], 0)
    part = size % P
    need, take, page, forked = _give(s, (part > 0).long())
    child = child & forked
    whole = (cols < (size // P)[:, None]) & child[:, None]
    _add_at(s["refcount"], table[at], whole, 1)
    last = (cols == (size // P)[:, None]) & (need > 0)[:, None]
    table.copy_(torch.where(last, page[:, :1], torch.where(whole, table[at], table)).to(torch.int32))
    s["row_pages"].copy_(torch.where(child, (size + P - 1) // P, s["row_pages"]).to(torch.int32))
    s["seq_len"].copy_(torch.where(child, size, s["seq_len"]))
    slot = torch.arange(P, device=DEV)
    which = ((slot[None, :] < part[:, None]) & (need > 0)[:, None]).view(-1).nonzero().view(-1)
    pos = ((size // P) * P)[:, None] + slot
    to, come = _places(table, pos, P).view(-1)[which], _places(table[at], pos, P).view(-1)[which]
    k, v = s["k"].view(L, -1, H, D), s["v"].view(L, -1, H, D)
    k[:, to] = k[:, come]
    v[:, to] = v[:, come]
    # reserve
    more = ((s["seq_len"] + s["extra"] + P - 1) // P - s["row_pages"]).clamp(min=0).long()
    need, take, page, granted = _give(s, more)
    held = s["row_pages"][:, None].long()
    mine = (cols >= held) & (cols < held + need[:, None])
    table.copy_(torch.where(mine, page.gather(1, (cols - held).clamp(min=0)), table).to(torch.int32))
    s["row_pages"].add_(need.to(torch.int32))
    return (s["k"], s["v"], table, s["row_pages"], s["seq_len"], s["refcount"],
            torch.stack([forked, granted]).to(torch.int32))


# ------------------------------------------------------------------- passes ---
def run(s):
    c = s["case"]
    if own:
        return _library(s, c["op"])
    if c["op"] == "attn":
        first = (lambda t: None if t is None else t[0])
        return _plain_attn(s["q"], s["k"], s["v"], s["table"], s["seq_len"], s["mask"], s["block_len"],
                           first(s.get("k_scale")), first(s.get("v_scale")))
    if c["op"] == "tree":
        return _plain_mask(s["parent"], s["block_len"]) + _plain_accept(s["parent"], s["tok"], s["top"][:, :, 0],
                                                                        s["block_len"])
    return _plain_cache(s) if c["op"] == "cache" else _plain_pages(s)


def _library(s, op):
    import draft_selection_amd as ds

    if op == "attn":
        scales = dict(k_scale=s["k_scale"][0], v_scale=s["v_scale"][0]) if "k_scale" in s else {}
        return ds.tree_attn(s["q"], s["k"], s["v"], s["table"], s["seq_len"], mask=s["mask"], block_len=s["block_len"],
                            out=s["out"], lse=s["lse"], **scales)
    if op == "tree":
        up = ds.tree_mask(s["parent"], block_len=s["block_len"], out=(s["mask"], s["depth"]))
        return tuple(up) + tuple(ds.tree_accept(s["parent"], s["tok"], s["top"][:, :, 0], block_len=s["block_len"]))
    if op == "cache":
        scales = dict(k_scale=s["k_scale"], v_scale=s["v_scale"]) if "k_scale" in s else {}
        ds.cache_append(s["k_new"], s["v_new"], s["k"], s["v"], s["table"], s["seq_len"], block_len=s["block_len"],
                        **scales)
        new_len = ds.cache_compact(s["k"], s["v"], s["table"], s["seq_len"], s["path"], s["n_keep"])
        return ((s["k"].float(), s["v"].float()) if scales else (s["k"], s["v"])) + (new_len,)
    pages = ds.Pages(s["table"], s["row_pages"], s["seq_len"], s["refcount"], s["case"]["page"])
    ds.pages_free(pages, s["which"])
    forked = ds.pages_fork(pages, s["src"], s["k"], s["v"])
    granted = ds.pages_reserve(pages, s["extra"])
    return (s["k"], s["v"], s["table"], s["row_pages"], s["seq_len"], s["refcount"], torch.cat([forked, granted]))


# ------------------------------------------------------------------- exact ---
def exact(c, seed):
    """The definition in 64 bits, sequence by sequence.  Outputs that are whole numbers, or copies of inputs, have none."""

    def attn(s):
        B, T, Hq, D = s["q"].shape
        P, H = c["page"], c["kv_heads"]
        out = torch.zeros((B, T, Hq, D), dtype=torch.float64, device=DEV)
        lse = torch.zeros((B, T, Hq), dtype=torch.float64, device=DEV)
        for b in range(B):
            done = int(s["seq_len"][b])
            n = int(s["block_len"][b]) if s["block_len"] is not None else T
            pages = s["table"][b, :(done + n + P - 1) // P].long()
            words = s["mask"][b, :n].cpu().tolist() if s["mask"] is not None else None
            rows = [[j <= i if words is None else (words[i][j // 32] >> (j % 32)) & 1 for j in range(n)] for i in range(n)]
            bias = torch.zeros((n, done + n), dtype=torch.float64, device=DEV)
            bias[:, done:] = torch.tensor([[0.0 if x else -math.inf for x in r] for r in rows], dtype=torch.float64)
            for h in range(H):
                K = s["k"][pages][:, :, h].reshape(-1, D)[:done + n].to(torch.float64)
                V = s["v"][pages][:, :, h].reshape(-1, D)[:done + n].to(torch.float64)
                if "k_scale" in s:
                    K, V = K * s["k_scale"][0, h].double(), V * s["v_scale"][0, h].double()
                for a in range(h * (Hq // H), (h + 1) * (Hq // H)):
                    z = torch.mm(s["q"][b, :n, a].to(torch.float64), K.T.contiguous()) / math.sqrt(D) + bias
                    lse[b, :n, a] = torch.logsumexp(z, dim=1)
                    out[b, :n, a] = torch.mm(torch.softmax(z, dim=1), V)
        return out, lse

    def written(s, n):
        """The 8-bit grid, value by value: 3 bits behind the leading one, down to steps of 2^-9."""
        cache = s[n].to(torch.float64)
        x = s[n + "_new"].to(torch.float64) / s[n + "_scale"].double()[:, None, None, :, None]
        step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
        x = (torch.round(x / step) * step).clamp(-448, 448)
        for b in range(c["B"]):
            m = int(s["block_len"][b]) if s["block_len"] is not None else c["T"]
            first, places = int(s["seq_len"][b]), s["table"][b].tolist()
            at = [(places[(first + t) // c["page"]], (first + t) % c["page"]) for t in range(c["T"])]
            for t in range(m):
                cache[:, at[t][0], at[t][1]] = x[:, b, t]
            for t, i in enumerate(s["path"][b, :int(s["n_keep"][b])].tolist()):
                cache[:, at[t][0], at[t][1]] = cache[:, at[i][0], at[i][1]].clone()
        return cache

    if c["op"] == "attn":
        return attn(prepare(c, seed))
    if c["op"] == "cache" and c["cache"] == "e4m3":
        s = prepare(c, seed)
        return written(s, "k"), written(s, "v"), None
    return None
