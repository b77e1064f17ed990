"""The operators of verifying drafts with a paged cache, in the cases that they are measured on.

The target's pass over a tree (or chain) of drafts attends, layer by layer, to the cache and to the
nodes on each node's own path (`tree_attention`).  Once the drafts are verified, the keys and values
of the accepted nodes of all layers go to the slots of the cache that were planned for them
(`append_path`).  Between rounds rows of the block tables are continued once or several times, or
freed: samples of one prompt, beams, finished requests (`fork_rows`).

`own` false: plain torch operations in 32 bits.  `own` true: the package's operators.
"""

import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}


def listed():
    return [
        # one stream with four drafts and the last token: what counts is the latency of a layer
        dict(name="tree_one_stream", op="tree", B=1, N=5, tree="chain", Hq=32, Hkv=8, D=128,
             page=16, dtype="bf16", len_lo=700, len_hi=700),
        # a batched round: trees of eleven nodes on 64 sequences of any length
        dict(name="tree_batch", op="tree", B=64, N=11, tree="binary", Hq=32, Hkv=8, D=128,
             page=16, dtype="bf16", len_lo=500, len_hi=8191),
        # wide trees: 256 (node, head) pairs to a key/value head
        dict(name="tree_wide", op="tree", B=32, N=64, tree="wide", Hq=32, Hkv=8, D=128,
             page=32, dtype="bf16", len_lo=500, len_hi=8191),
        # two sequences with a very long context each
        dict(name="tree_long", op="tree", B=2, N=16, tree="chain", Hq=32, Hkv=8, D=128,
             page=64, dtype="bf16", len_lo=131000, len_hi=131072),
        # short and empty caches, pages that are no power of two, seven heads to a shared one
        dict(name="tree_uneven_f16", op="tree", B=19, N=13, tree="comb", Hq=28, Hkv=4, D=64,
             page=20, dtype="f16", len_lo=0, len_hi=1333),
        # no drafts: one token of each of 256 sequences
        dict(name="tree_decode", op="tree", B=256, N=1, tree="chain", Hq=32, Hkv=8, D=128,
             page=64, dtype="bf16", len_lo=200, len_hi=8000),
        # one stream's accepted drafts, in the caches of 32 layers
        dict(name="append_one_stream", op="append", B=1, N=5, tree="chain", L=32, Hkv=8, D=128,
             page=16, dtype="bf16", len_hi=700, none=0.0),
        # a batched round with trees
        dict(name="append_batch", op="append", B=64, N=11, tree="binary", L=32, Hkv=8, D=128,
             page=16, dtype="bf16", len_hi=200, none=0.1),
        # many sequences, wide trees, pages that are no power of two, float32
        dict(name="append_wide_f32", op="append", B=256, N=40, tree="wide", L=12, Hkv=4, D=80,
             page=20, dtype="f32", len_hi=100, none=0.3),
        # eight samples of one prompt
        dict(name="fork_samples", op="fork", S=1, B=8, L=32, Hkv=8, D=128, page=16, dtype="bf16",
             len_lo=1503, len_hi=1503, spare=3, gone=0.0, forks=7 / 8, shared=0, short=False),
        # beams of a batch after a step: some continued several times, some not at all
        dict(name="fork_beams", op="fork", S=64, B=64, L=8, Hkv=8, D=128, page=16, dtype="bf16",
             len_lo=300, len_hi=1200, spare=2, gone=0.05, forks=0.4, shared=20, short=False),
        # a large batch with long tables: one row in ten ends, one in four is new
        dict(name="fork_large", op="fork", S=512, B=512, L=4, Hkv=2, D=128, page=64, dtype="bf16",
             len_lo=0, len_hi=9000, spare=1, gone=0.1, forks=0.25, shared=10, short=False),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("tree", "tree", "tree", "append", "fork"))
    Hkv = rng.choice((1, 2, 4, 8))
    page = rng.choice((5, 16, 16, 20, 32, 64, 128))
    if op == "tree":
        B, N, D = _spread(rng, 1, 256), _spread(rng, 1, 64), rng.choice((64, 128, 128, 256))
        Hq = Hkv * rng.choice((1, 3, 4, 7, 8))
        # as many cached tokens as keep bytes and products below the largest listed case's
        most = min(131072, 2 * 10 ** 9 // (2 * B * Hkv * D), 10 ** 11 // (4 * B * N * Hq * D))
        hi = _spread(rng, 1, max(2, most))
        return dict(op=op, B=B, N=N, tree=rng.choice(("chain", "binary", "wide", "comb")), Hq=Hq,
                    Hkv=Hkv, D=D, page=page, dtype=rng.choice(("bf16", "f16")),
                    len_lo=rng.choice((0, hi // 2, hi)), len_hi=hi)
    D = rng.choice((64, 80, 128, 256))
    dtype = rng.choice(("bf16", "bf16", "f16", "f32"))
    row = Hkv * D * BYTES[dtype]
    if op == "append":
        B, N = _spread(rng, 1, 256), _spread(rng, 1, 64)
        hi = _spread(rng, 1, 200)
        room = row * B * (2 * hi + 2 * N + page)  # of a layer: caches and nodes
        return dict(op=op, B=B, N=N, tree=rng.choice(("chain", "binary", "wide", "comb")),
                    L=_spread(rng, 1, max(1, min(48, 10 ** 9 // room))), Hkv=Hkv, D=D, page=page,
                    dtype=dtype, len_hi=hi, none=rng.choice((0.0, 0.3)))
    S = _spread(rng, 1, 512)
    B = min(512, S * rng.choice((1, 1, 2, 8)))
    hi = _spread(rng, 1, max(2, min(20000, 8 * 10 ** 8 // (row * S))))
    room = row * (S * (hi + 4 * page) + B * page)  # of a layer
    return dict(op=op, S=S, B=B, L=_spread(rng, 1, max(1, min(32, 10 ** 9 // room))), Hkv=Hkv,
                D=D, page=page, dtype=dtype, len_lo=rng.choice((0, hi // 2, hi)), len_hi=hi,
                spare=rng.randint(0, 3), gone=rng.choice((0.0, 0.1)),
                forks=rng.choice((0.0, 0.3, 0.7)), shared=rng.choice((0, 15)),
                short=rng.random() < 0.2)


def _parents(tree, N):
    """parent[u] < u of each node; node 0, the last token, is the root."""
    if tree == "chain":
        return np.arange(-1, N - 1)
    if tree == "binary":
        return (np.arange(N) - 1) // 2 if N else np.arange(0)
    if tree == "wide":
        return (np.arange(N) - 1) // 4
    # "comb": every odd node goes on from the odd node before, even ones are leaves beside it
    u = np.arange(N)
    return np.where(u == 0, -1, np.where(u % 2 == 1, np.maximum(u - 2, 0), np.maximum(u - 3, 0)))


def _paths(parent):
    """path[u, v]: whether node v lies on the way from the root to node u, u included."""
    path = np.eye(len(parent), dtype=bool)
    for u in range(1, len(parent)):
        path[u] |= path[parent[u]]
    return path


def _depths(parent):
    return _paths(parent).sum(1) - 1


def _accepted(case):
    """Tokens that each sequence adds: the last one and the nodes accepted after it, any number
    up to the tree's depth; none for sequences that have no pages."""
    depth = int(_depths(_parents(case["tree"], case["N"])).max())
    new = 1 + _even(0, depth, case["B"])
    every = round(1 / case["none"]) if case["none"] else 0
    if every:
        new[every - 1::every] = 0
    return new


def _even(lo, hi, n):
    """n whole numbers spread evenly over [lo, hi]."""
    return np.linspace(lo, hi, n).round().astype(np.int64)


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def _table(count, ids, cols, rest):
    """Rows of page ids, `count` in each, and `rest` behind them."""
    t = np.full((len(count), cols), rest, dtype=np.int64)
    t[np.arange(cols) < count[:, None]] = ids[:int(count.sum())]
    return t


def _normal(shape, dtype, gen):
    return torch.empty(shape, dtype=DTYPES[dtype], device="cuda").normal_(generator=gen)


# ---- attention of the nodes: a layer's queries, keys and values, and the cache ------------------


def _prepare_tree(case, seed):
    rng = np.random.default_rng(seed)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    B, N, P, Hq, Hkv, D = (case[k] for k in ("B", "N", "page", "Hq", "Hkv", "D"))
    lens = rng.permutation(_even(case["len_lo"], case["len_hi"], B))
    pages = -(-lens // P)
    ids = rng.permutation(int(pages.sum()) + 3)
    # queries, keys and values are pieces of one projection
    qkv = _normal((B, N, Hq + 2 * Hkv, D), case["dtype"], gen)
    shape = (len(ids), P, Hkv, D)
    return dict(q=qkv[:, :, :Hq], k=qkv[:, :, Hq:Hq + Hkv], v=qkv[:, :, Hq + Hkv:],
                k_cache=_normal(shape, case["dtype"], gen),
                v_cache=_normal(shape, case["dtype"], gen),
                tables=_i32(_table(pages, ids, max(1, int(pages.max())), 0)), lens=_i32(lens),
                most=int(lens.max()), parent=_parents(case["tree"], N).astype(np.int32),
                scale=D ** -0.5)


def _plain_tree(s):
    q, most = s["q"], s["most"]
    B, N, Hq, D = q.shape
    P, Hkv = s["k_cache"].shape[1:3]
    dev = q.device
    t = torch.arange(most, device=dev)
    cached = (t < s["lens"][:, None])[:, None].expand(B, N, most)
    nodes = torch.from_numpy(_paths(s["parent"])).to(dev).expand(B, N, N)
    ok = torch.cat([cached, nodes], 2)[:, None, :, None]           # [B, 1, N, 1, tokens]

    def tokens(cache, new):
        old = cache[s["tables"][:, t // P].long(), t % P]
        return torch.cat([old, new], 1).permute(0, 2, 1, 3).float()  # [B, Hkv, tokens, D]

    x = q.float().view(B, N, Hkv, Hq // Hkv, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, -1, D)
    score = (x @ tokens(s["k_cache"], s["k"]).transpose(-1, -2)) * s["scale"]
    score = score.view(B, Hkv, N, Hq // Hkv, -1)
    score = torch.where(ok, score, -math.inf)
    top = score.amax(-1, keepdim=True)                               # a node sees itself
    w = torch.exp(score - top)
    total = w.sum(-1, keepdim=True)
    out = w.view(B, Hkv, -1, most + N) @ tokens(s["v_cache"], s["v"])
    out = out.view(B, Hkv, N, -1, D) / total
    lse = (top + torch.log(total))[..., 0]
    return {"out": out.permute(0, 2, 1, 3, 4).reshape(B, N, Hq, D).to(q.dtype),
            "lse": lse.permute(0, 2, 1, 3).reshape(B, N, Hq)}


def _own_tree(s):
    import sampling_ssd_verify_gb300 as ssd

    o = ssd.tree_attention(s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"], s["tables"],
                           s["lens"], parent=s["parent"], scale=s["scale"], out=s["out"])
    return {"out": o["out"], "lse": o["lse"]}


def _exact_tree(s):
    """Sequence by sequence, the nodes' scores beside the cached tokens', in float64."""
    B, N, Hq, D = s["q"].shape
    Hkv = s["k"].shape[2]
    M = Hq // Hkv
    out = torch.empty((B, N, Hq, D), dtype=torch.float64, device="cuda")
    lse = torch.empty((B, N, Hq), dtype=torch.float64, device="cuda")
    parent = s["parent"].tolist()
    sees = torch.zeros((N, N), dtype=torch.bool)
    for u in range(N):
        v = u
        while v >= 0:
            sees[u, v] = True
            v = parent[v]
    hidden = ~sees.cuda()[None, :, None]
    P = s["k_cache"].shape[1]
    for b, n in enumerate(s["lens"].tolist()):
        held = s["tables"][b, :-(-n // P)].long()
        for h in range(Hkv):
            x = s["q"][b, :, h * M:(h + 1) * M].double()
            k, v = (torch.cat([c[held, :, h].reshape(-1, D)[:n], a[b, :, h]]).double()
                    for c, a in ((s["k_cache"], s["k"]), (s["v_cache"], s["v"])))
            sc = torch.einsum("umd,td->umt", x, k) * s["scale"]
            sc[..., n:].masked_fill_(hidden[0], -math.inf)
            out[b, :, h * M:(h + 1) * M] = torch.einsum("umt,td->umd", torch.softmax(sc, -1), v)
            lse[b, :, h * M:(h + 1) * M] = torch.logsumexp(sc, -1)
    return {"out": out, "lse": lse}


# ---- accepted nodes into the caches: verification's paths and the plan of the new tokens --------


def _prepare_append(case, seed):
    rng = np.random.default_rng(seed)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    B, N, P, L, Hkv, D = (case[k] for k in ("B", "N", "page", "L", "Hkv", "D"))
    parent = _parents(case["tree"], N)
    depth = _depths(parent)
    path = np.full((B, max(1, int(depth.max()))), -1, dtype=np.int64)
    new = rng.permutation(_accepted(case))
    for b in range(B):  # the way to a node of that depth
        u = int(rng.choice(np.nonzero(depth == max(0, new[b] - 1))[0]))
        while u > 0:
            path[b, depth[u] - 1] = u
            u = parent[u]
    lens = rng.permutation(_even(0, case["len_hi"], B))
    pages = -(-(lens + new) // P)
    ids = rng.permutation(int((-(-(lens + 1 + depth.max()) // P)).sum()) + 3)
    table = _table(pages, ids, max(1, int(pages.max())), -1)
    cu = np.concatenate([[0], new.cumsum()])
    rows = B * (1 + int(depth.max()))
    owner, slots = np.full(rows, -1), np.full(rows, -1)
    T = int(cu[-1])
    owner[:T] = np.repeat(np.arange(B), new)
    pos = lens[owner[:T]] + np.arange(T) - cu[owner[:T]]
    slots[:T] = table[owner[:T], pos // P] * P + pos % P
    dt = case["dtype"]
    return dict(k=_normal((L, B, N, Hkv, D), dt, gen), v=_normal((L, B, N, Hkv, D), dt, gen),
                k_cache=_normal((L, len(ids), P, Hkv, D), dt, gen),
                v_cache=_normal((L, len(ids), P, Hkv, D), dt, gen),
                slots=torch.from_numpy(slots.astype(np.int64)).cuda(), owner=_i32(owner),
                cu=_i32(cu), path=_i32(path))


def _plain_append(s):
    P = s["k_cache"].shape[2]
    slots, b = s["slots"], s["owner"].long().clamp(min=0)
    i = torch.arange(len(slots), device="cuda") - s["cu"][b]
    node = torch.where(i > 0, s["path"][b, (i - 1).clamp(0, s["path"].shape[1] - 1)].long(), 0)
    live = slots >= 0
    slots, b, node = slots[live], b[live], node[live]
    for cache, new in ((s["k_cache"], s["k"]), (s["v_cache"], s["v"])):
        cache[:, slots // P, slots % P] = new[:, b, node]
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _own_append(s):
    import sampling_ssd_verify_gb300 as ssd

    ssd.append_path(s["k"], s["v"], s["k_cache"], s["v_cache"], s["slots"], s["owner"], s["cu"],
                    s["path"])
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _exact_append(s):
    """Token by token."""
    P = s["k_cache"].shape[2]
    cu, path = s["cu"].tolist(), s["path"].tolist()
    slots = s["slots"].tolist()
    for b in range(len(cu) - 1):
        nodes = [0] + path[b]
        for i, t in enumerate(range(cu[b], cu[b + 1])):
            at = divmod(slots[t], P)
            s["k_cache"][:, at[0], at[1]] = s["k"][:, b, nodes[i]]
            s["v_cache"][:, at[0], at[1]] = s["v"][:, b, nodes[i]]
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _continued(case):
    """How many old rows go on, and how often one is forked."""
    rows = case["B"] - int(case["gone"] * case["B"])
    heirs = max(1, min(case["S"], rows - int(case["forks"] * rows)))
    return heirs, rows - heirs


# ---- rows continued, shared and freed ------------------------------------------------------------


def _prepare_fork(case, seed):
    rng = np.random.default_rng(seed)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    S, B, P, L, Hkv, D = (case[k] for k in ("S", "B", "page", "L", "Hkv", "D"))
    lens = rng.permutation(_even(case["len_lo"], case["len_hi"], S))
    held = -(-lens // P) + rng.integers(0, case["spare"] + 1, S)
    # one row in two has its first full pages in common with the row before it
    common = np.where(np.arange(S) % 2 == 1, np.minimum(lens, np.roll(lens, 1)) // P, 0)
    common = np.minimum(common, case["shared"])
    own_pages = held - common
    heirs, forks = _continued(case)
    src = np.full(B, -1)
    src[:heirs] = rng.permutation(S)[:heirs]
    src[heirs:heirs + forks] = rng.choice(src[:heirs], forks)
    src = rng.permutation(src)
    free = forks // 3 if case["short"] else forks + 5
    pool = int((-(-lens // P) + case["spare"]).sum()) + free  # some belong to nobody here
    ids = rng.permutation(pool)
    table = np.full((S, max(1, -(-case["len_hi"] // P) + case["spare"])), -1, dtype=np.int64)
    at = free
    shares = np.zeros(pool, dtype=np.int64)
    for r in range(S):
        c, n = int(common[r]), int(own_pages[r])
        if c:
            table[r, :c] = table[r - 1, :c]
            shares[table[r, :c]] += 1
        table[r, c:c + n] = ids[at:at + n]
        at += n
    stack = np.full(pool, -1, dtype=np.int64)
    stack[:free] = ids[:free]
    dt = case["dtype"]
    return dict(src=_i32(src), lens=_i32(lens), held=_i32(held), tables=_i32(table),
                shares=_i32(shares), free_pages=_i32(stack), free_count=_i32([free]), page=P,
                k_cache=_normal((L, pool, P, Hkv, D), dt, gen),
                v_cache=_normal((L, pool, P, Hkv, D), dt, gen))


def _plain_fork(s):
    P = s["page"]
    src, lens, held = (s[k].long() for k in ("src", "lens", "held"))
    tables, stack, n = s["tables"].long(), s["free_pages"].clone(), s["free_count"].long()
    S, W = tables.shape
    B, dev = len(src), src.device
    row, col, ent = (torch.arange(m, device=dev) for m in (B, W, S * W))
    goes = src >= 0
    at = torch.where(goes, src, S)
    heir = torch.full((S + 1,), B, device=dev).scatter_reduce(0, at, row, "amin")
    first = goes & (heir[at] == row)
    # pages of rows that nobody continues: the last holder of a page gives it back
    ends = (heir[:S] == B)[:, None] & (col < held[:, None])
    pool = len(s["shares"])
    page = torch.where(ends, tables, pool).view(-1)
    shares = torch.cat([s["shares"].long(), held.new_zeros(1)])
    shares = shares.scatter_add(0, page, torch.full_like(page, -1))
    last = torch.full((pool + 1,), -1, device=dev).scatter_reduce(0, page, ent, "amax")
    back = ends.view(-1) & (shares[page] < 0) & (last[page] == ent)
    order = back.cumsum(0) - 1
    put = torch.where(back, n + order, len(stack))
    stack = torch.cat([stack, stack.new_zeros(1)]).scatter(0, put, page.int())[:-1]
    top = n + back.sum()
    shares = shares[:-1].clamp(min=0)
    # the others share the full pages and take one for the last
    full, part = lens // P, lens % P
    from_ = src.clamp(min=0)
    more = goes & ~first
    takes = more & (part[from_] > 0)
    nth = takes.cumsum(0) - 1
    served = ~takes | (nth < top)
    live = goes & served
    fresh = stack[(top - 1 - nth).clamp(0, len(stack) - 1)].long()
    out_len = torch.where(live, lens[from_], 0)
    kept = torch.where(first, held[from_], full[from_] + (part[from_] > 0).long())
    out_held = torch.where(live, kept, 0)
    out = torch.where(col < out_held[:, None], tables[from_], -1)
    takes = takes & served
    out = torch.where(takes[:, None] & (col == full[from_][:, None]), fresh[:, None], out)
    join = (more & served)[:, None] & (col < full[from_][:, None])
    joined = torch.where(join, tables[from_], pool).view(-1)
    shares = torch.cat([shares, shares.new_zeros(1)])
    shares = shares.scatter_add(0, joined, torch.ones_like(joined))[:-1]
    # tokens of the last pages
    b = takes.nonzero()[:, 0]
    old, new = tables[src[b], full[src[b]].clamp(max=W - 1)], fresh[b]
    there = (torch.arange(P, device=dev) < part[src[b]][:, None])[..., None, None]
    for cache in (s["k_cache"], s["v_cache"]):
        cache[:, new] = torch.where(there, cache[:, old], cache[:, new])
    return {"tables": out.int(), "lens": out_len.int(), "held": out_held.int(),
            "served": served.int(), "shares": shares.int(),
            "free_count": (top - takes.sum()).int(), "free_pages": stack,
            "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _own_fork(s):
    import sampling_ssd_verify_gb300 as ssd

    o = ssd.fork_rows(s["src"], s["lens"], s["held"], s["tables"], s["shares"], s["free_pages"],
                      s["free_count"], s["page"], s["k_cache"], s["v_cache"], out=s["out"])
    o = {k: o[k] for k in ("tables", "lens", "held", "served", "shares", "free_count")}
    return dict(o, free_pages=s["free_pages"], k_cache=s["k_cache"], v_cache=s["v_cache"])


def _exact_fork(s):
    """Row by row, with Python lists."""
    P = s["page"]
    src, lens, held, shares = (s[k].tolist() for k in ("src", "lens", "held", "shares"))
    tables, rest = s["tables"].tolist(), s["free_pages"].tolist()
    W = len(tables[0])
    n = int(s["free_count"])
    stack = rest[:n]
    holders = [x + 1 for x in shares]
    lost = [(r, c) for r in range(len(lens)) if r not in set(src) for c in range(held[r])]
    for r, c in lost:
        p = tables[r][c]
        holders[p] -= 1
        if holders[p] == 0:
            stack.append(p)
    pushed = stack + rest[len(stack):]
    o = dict(tables=[], lens=[], held=[], served=[])
    seen = set()
    for r in src:
        pages, length, ok = [], 0, 1
        if r >= 0 and r not in seen:
            seen.add(r)
            pages, length = tables[r][:held[r]], lens[r]
        elif r >= 0:
            whole, tail = divmod(lens[r], P)
            if tail and not stack:
                ok = 0
            else:
                pages, length = tables[r][:whole], lens[r]
                for p in pages:
                    holders[p] += 1
                if tail:
                    p = stack.pop()
                    holders[p] = 1
                    for c in (s["k_cache"], s["v_cache"]):
                        c[:, p, :tail] = c[:, tables[r][whole], :tail]
                    pages = pages + [p]
        o["tables"].append(pages + [-1] * (W - len(pages)))
        o["lens"].append(length)
        o["held"].append(len(pages))
        o["served"].append(ok)
    o = {k: torch.tensor(v) for k, v in o.items()}
    return dict(o, shares=torch.tensor([max(0, x - 1) for x in holders]),
                free_count=torch.tensor([len(stack)]), free_pages=torch.tensor(pushed),
                k_cache=s["k_cache"], v_cache=s["v_cache"])


# ---- what the tools call --------------------------------------------------------------------------


def prepare(case, seed):
    """The inputs, and `out`: where a program that calls again and again keeps the outputs."""
    make = {"tree": _prepare_tree, "append": _prepare_append, "fork": _prepare_fork}[case["op"]]
    return dict(make(case, seed), op=case["op"], out={})


def run(state):
    op = state["op"]
    if op == "tree":
        return _own_tree(state) if own else _plain_tree(state)
    if op == "append":
        return _own_append(state) if own else _plain_append(state)
    return _own_fork(state) if own else _plain_fork(state)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "tree":
        return _exact_tree(s)
    if case["op"] == "append":
        return _exact_append(s)
    return _exact_fork(s)


def work(case):
    Hkv, D, es = case["Hkv"], case["D"], BYTES[case["dtype"]]
    if case["op"] == "tree":
        B, N, Hq = case["B"], case["N"], case["Hq"]
        cached = int(_even(case["len_lo"], case["len_hi"], B).sum())
        pairs = N * cached + B * int(_paths(_parents(case["tree"], N)).sum())
        b = es * D * (2 * B * N * Hq + 2 * Hkv * (cached + B * N)) + 4 * B * N * Hq
        return {"bytes": b + 4 * (cached // case["page"] + B), "flops": 4 * Hq * D * pairs}
    if case["op"] == "append":
        T = int(_accepted(case).sum())
        return {"bytes": T * (4 * case["L"] * Hkv * D * es + 16) + 8 * case["B"], "flops": 0}
    S, B, P = case["S"], case["B"], case["page"]
    lens = _even(case["len_lo"], case["len_hi"], S)
    heirs, forks = _continued(case)
    # a fork copies the tokens of its last page, while there are pages
    tokens = (forks // 3 if case["short"] else forks) * float((lens % P).mean())
    pages = float((-(-lens // P)).mean())
    return {"bytes": tokens * 4 * case["L"] * Hkv * D * es + 4 * pages * (S + heirs + forks)
            + 8 * (pages * S + forks) + 4 * (2 * S + 4 * B), "flops": 0}
