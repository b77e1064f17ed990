"""The operators around a round of speculative decoding, in the cases that they are measured on.

Before a round the target's logits of every draft position are adjusted for repeated tokens,
biases and a grammar (`process_logits`).  After it the accepted lengths decide which pages of the
key/value cache every request holds and where its next tokens go (`page_plan`).  While the target
works, the branches of the outcome cache are continued: all branches of a sequence share its
prefix and have a few tokens of their own (`prefix_attention`).

`own` false: plain torch operations in 32 bits.  `own` true: the package's operators.
"""

import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}
FILL = -math.inf  # what a token outside the grammar gets

# Drafts as trees: the parent of each node (a chain where a case names none).
TREES = {"uneven-11": (-1, 0, 0, 1, 1, 1, 2, 4, 4, 7, 8),
         "binary-depth-3": (-1, 0, 0, 1, 1, 2, 2)}


def listed():
    return [
        # one stream with four drafts: what counts is the time until the round can start
        dict(name="logits_one_stream", op="logits", B=1, N=5, V=128256, dtype="bf16", tree="",
             history=700, biases=16, grammar=True),
        # the batched round: 64 sequences, eight drafts, half of them under a grammar
        dict(name="logits_batch_bf16", op="logits", B=64, N=9, V=128256, dtype="bf16", tree="",
             history=2048, biases=64, grammar=True),
        # the largest round, float32 logits, long histories
        dict(name="logits_large_f32", op="logits", B=256, N=9, V=151936, dtype="f32", tree="",
             history=4096, biases=300, grammar=True),
        # tree drafts over an odd vocabulary (rows start at any alignment), penalties alone
        dict(name="logits_tree_odd", op="logits", B=37, N=11, V=50257, dtype="bf16",
             tree="uneven-11", history=1111, biases=0, grammar=False),
        # a round's bookkeeping: 32 sequences, four drafts and the bonus token
        dict(name="pages_round", op="pages", B=32, page=16, new_lo=5, new_hi=5, most=8000,
             spare=5, short=False),
        # 256 sequences of any length, some of them idle, pages of 64 tokens
        dict(name="pages_batch", op="pages", B=256, page=64, new_lo=0, new_hi=9, most=32000,
             spare=80, short=False),
        # prompts come in beside running requests, and the pool has fewer pages than they ask for
        dict(name="pages_prompts", op="pages", B=1000, page=16, new_lo=1, new_hi=1023, most=4000,
             spare=40, short=True),
        # twelve branches of one sequence
        dict(name="attn_one_stream", op="attn", G=1, n_lo=12, n_hi=12, Hq=32, Hkv=8, D=128,
             page=16, dtype="bf16", pre_lo=1500, pre_hi=1500, suf_lo=1, suf_hi=4),
        # the cache build: twelve branches of each of 32 sequences
        dict(name="attn_cache_build", op="attn", G=32, n_lo=12, n_hi=12, Hq=32, Hkv=8, D=128,
             page=16, dtype="bf16", pre_lo=500, pre_hi=8191, suf_lo=1, suf_hi=4),
        # 24 branches of each of 256 sequences
        dict(name="attn_large_batch", op="attn", G=256, n_lo=24, n_hi=24, Hq=32, Hkv=8, D=128,
             page=64, dtype="bf16", pre_lo=200, pre_hi=2000, suf_lo=1, suf_hi=8),
        # one long common prompt for 256 requests that have gone on by themselves
        dict(name="attn_common_prompt", op="attn", G=1, n_lo=256, n_hi=256, Hq=32, Hkv=8, D=128,
             page=32, dtype="bf16", pre_lo=16000, pre_hi=16000, suf_lo=0, suf_hi=900),
        # uneven groups, empty prefixes and suffixes, seven heads to a shared one, odd pages
        dict(name="attn_uneven_f16", op="attn", G=19, n_lo=1, n_hi=9, Hq=28, Hkv=4, D=64,
             page=20, dtype="f16", pre_lo=0, pre_hi=1333, suf_lo=0, suf_hi=70),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("logits", "logits", "pages", "attn", "attn", "attn"))
    if op == "logits":
        tree = rng.choice(("", "", "uneven-11", "binary-depth-3"))
        N = len(TREES[tree]) if tree else rng.randint(1, 9)
        dtype = rng.choice(("bf16", "f32"))
        V = _spread(rng, 1000, 152000)
        most = 256 * 9 * 151936 * 4 // (N * V * BYTES[dtype])
        return dict(op=op, B=_spread(rng, 1, min(256, most)), N=N, V=V, dtype=dtype, tree=tree,
                    history=_spread(rng, 1, 4096), biases=rng.choice((0, 1, 17, 300)),
                    grammar=rng.random() < 0.6)
    if op == "pages":
        lo = rng.randint(0, 9)
        return dict(op=op, B=_spread(rng, 1, 1000), page=rng.choice((1, 8, 16, 20, 64, 128)),
                    new_lo=lo, new_hi=lo + _spread(rng, 1, 1000) - 1, most=_spread(rng, 1, 4000),
                    spare=rng.randint(0, 90), short=rng.random() < 0.3)
    G = _spread(rng, 1, 256)
    Hkv = rng.choice((1, 2, 4, 8))
    n_hi = max(1, min(_spread(rng, 1, 64), 6144 // G))
    longest = min(16000, 256 * 1100 * 8 // (G * Hkv))
    pre = _spread(rng, 1, longest)
    suf = min(rng.choice((0, 4, 8, 100, 900)), 230400 // (G * n_hi))
    return dict(op=op, G=G, n_lo=rng.randint(1, n_hi), n_hi=n_hi,
                Hq=Hkv * rng.choice((1, 3, 4, 7, 8)), Hkv=Hkv, D=rng.choice((64, 128, 128, 256)),
                page=rng.choice((5, 16, 20, 32, 64, 128)), dtype=rng.choice(("bf16", "f16")),
                pre_lo=rng.choice((0, pre // 2, pre)), pre_hi=pre,
                suf_lo=rng.choice((0, suf)), suf_hi=suf)


def _even(lo, hi, n):
    """n whole numbers spread evenly over [lo, hi]."""
    return np.linspace(lo, hi, n).round().astype(np.int64)


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


# ---- logits: what a sampler's program has before the round ------------------------------------


def _prepare_logits(case, seed):
    B, N, V = case["B"], case["N"], case["V"]
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rng = np.random.default_rng(seed)
    logits = torch.empty((B, N, V), dtype=DTYPES[case["dtype"]], device="cuda")
    for b in range(0, B, 32):  # in pieces, so that large batches need little room
        part = torch.randn((min(32, B - b), N, V), generator=gen, device="cuda") * 2.5
        logits[b:b + 32] = part.to(logits.dtype)
    H = case["history"]
    # few tokens are frequent and many rare, each sequence with its own
    rank = np.minimum(V - 1, np.floor(V ** rng.random((B, H)) - 1)).astype(np.int64)
    history = (rank * 7919 + rng.integers(0, V, (B, 1))) % V
    length = rng.permutation(_even(H // 2, H, B))
    tree = case["tree"]
    drafts = rng.integers(0, V, (B, N if tree else N - 1))
    if drafts.size:  # one draft in three repeats a token of the history
        again = rng.random(drafts.shape) < 0.33
        drafts = np.where(again, np.take_along_axis(history, rng.integers(0, H, drafts.shape), 1), drafts)
    s = dict(logits=logits, history=_i32(history), history_len=_i32(length),
             prompt_len=_i32(length // 2), drafts=_i32(drafts),
             parent=np.asarray(TREES[tree] if tree else range(-1, N - 1), dtype=np.int32),
             repetition=torch.from_numpy(rng.uniform(1.0, 1.4, B).astype(np.float32)).cuda(),
             presence=torch.from_numpy(rng.uniform(0.0, 1.0, B).astype(np.float32)).cuda(),
             frequency=torch.from_numpy(rng.uniform(0.0, 0.5, B).astype(np.float32)).cuda(),
             bias_ids=None, bias=None, mask=None)
    if case["biases"]:
        nb = min(case["biases"], V)
        s["bias_ids"] = _i32((rng.permutation(V)[None, :nb] + rng.integers(0, V, (B, 1))) % V)
        s["bias"] = torch.from_numpy(rng.uniform(-4, 4, (B, nb)).astype(np.float32)).cuda()
    if case["grammar"]:
        words = [torch.randint(-2 ** 31, 2 ** 31, (B, N, (V + 31) // 32), generator=gen,
                               device="cuda", dtype=torch.int64).to(torch.int32) for _ in range(2)]
        mask = words[0] & words[1]
        mask[::2] = -1  # every other sequence is free
        if B > 1:
            mask[1, 0] = 0  # and one row has reached a dead end
        s["mask"] = mask
    return s


def _plain_logits(s):
    logits, parent = s["logits"], s["parent"]
    B, N, V = logits.shape
    dev = logits.device
    place = torch.arange(s["history"].shape[1], device=dev)
    valid = place < s["history_len"][:, None]
    said = valid & (place >= s["prompt_len"][:, None])
    ids = s["history"].long()
    seen = torch.zeros((B, V), device=dev).scatter_add_(1, ids, valid.float())
    count = torch.zeros((B, V), device=dev).scatter_add_(1, ids, said.float())
    # the drafts on the path to each row
    path = _paths(parent)
    row, node = np.nonzero(path[:, 1:])
    more = torch.zeros((B, N, V), device=dev)
    if row.size:
        drafts = s["drafts"][:, -(N - 1):].long()  # a tree's tokens have an entry for its root
        at = torch.from_numpy(row * V).to(dev) + drafts[:, torch.from_numpy(node).to(dev)]
        more.view(B, N * V).scatter_add_(1, at, torch.ones(at.shape, device=dev))
    seen = (seen[:, None] + more) > 0
    count = count[:, None] + more
    z = logits.float()
    r = s["repetition"][:, None, None]
    z = torch.where(seen, torch.where(z > 0, z / r, z * r), z)
    z = z - s["frequency"][:, None, None] * count - s["presence"][:, None, None] * (count > 0)
    if s["bias"] is not None:
        z = z + torch.zeros((B, V), device=dev).scatter_(1, s["bias_ids"].long(), s["bias"])[:, None]
    if s["mask"] is None:
        return {"logits": z.to(logits.dtype)}
    v = torch.arange(V, device=dev)
    ok = ((s["mask"][..., v // 32] >> (v % 32).to(torch.int32)) & 1).bool()
    return {"logits": torch.where(ok, z, FILL).to(logits.dtype),
            "allowed": ok.sum(-1, dtype=torch.int32)}


def _paths(parent):
    """path[u, v]: whether node v lies on the way from the root to node u, u included."""
    N = len(parent)
    path = np.eye(N, dtype=bool)
    for u in range(1, N):
        path[u] |= path[parent[u]]
    return path


def _own_logits(s):
    import sampling_ssd_verify_gb300 as ssd

    return ssd.process_logits(s["logits"], s["history"], s["history_len"], s["prompt_len"],
                              draft_tokens=s["drafts"], parent=s["parent"],
                              repetition=s["repetition"], presence=s["presence"],
                              frequency=s["frequency"], bias_ids=s["bias_ids"], bias=s["bias"],
                              mask=s["mask"], fill=FILL, allowed=s["mask"] is not None,
                              out=s["out"])


def _exact_logits(s):
    """Sequence by sequence, in float64."""
    B, N, V = s["logits"].shape
    parent = s["parent"].tolist()
    tokens = s["drafts"].tolist()
    outs, allowed = [], []
    bit = torch.arange(32, device="cuda")
    for b in range(B):
        n, m = int(s["history_len"][b]), int(s["prompt_len"][b])
        h = s["history"][b, :n].long()
        prompt = torch.bincount(h[:m], minlength=V).double()
        spoken = torch.bincount(h[m:], minlength=V).double()
        r, a, f = (s[k][b].double() for k in ("repetition", "presence", "frequency"))
        z = s["logits"][b].double()
        for u in range(N):
            c = spoken.clone()
            w = u
            while w > 0:
                c[tokens[b][w if len(tokens[b]) == N else w - 1]] += 1
                w = parent[w]
            hit = (prompt + c) > 0
            x = z[u]
            x = torch.where(hit & (x > 0), x / r, torch.where(hit, x * r, x))
            x = x - f * c
            x = torch.where(c > 0, x - a, x)
            if s["bias"] is not None:
                x[s["bias_ids"][b].long()] += s["bias"][b].double()
            if s["mask"] is not None:
                ok = ((s["mask"][b, u].long()[:, None] >> bit) & 1).reshape(-1)[:V] == 1
                x = torch.where(ok, x, torch.full_like(x, FILL))
                allowed.append(int(ok.sum()))
            z[u] = x
        outs.append(z)
    out = {"logits": torch.stack(outs)}
    if s["mask"] is not None:
        out["allowed"] = torch.tensor(allowed, dtype=torch.int64).view(B, N)
    return out


# ---- pages: lengths after a round, the tables so far and the free pages -----------------------


def _prepare_pages(case, seed):
    rng = np.random.default_rng(seed)
    B, P = case["B"], case["page"]
    lens = rng.permutation(_even(0, case["most"], B))
    new = rng.permutation(_even(case["new_lo"], case["new_hi"], B))
    held = -(-(lens + rng.integers(0, case["spare"] + 1, B)) // P)  # pages of drafts not taken
    need = -(-(lens + new) // P)
    ask, back = np.maximum(need - held, 0).sum(), np.maximum(held - need, 0).sum()
    free = max(0, int(ask * (0.8 if case["short"] else 1.5)) - int(back)) + (0 if case["short"] else 7)
    W = 1 - (-(case["most"] + max(case["spare"], case["new_hi"])) // P)
    pages = rng.permutation(int(held.sum()) + free)
    tables = np.full((B, W), -1, dtype=np.int64)
    cols = np.arange(W) < held[:, None]
    tables[cols] = pages[free:]
    room = 8 + 2 * B * (3 + case["new_hi"] // P + case["spare"] // P)
    stack = np.full(room, -1, dtype=np.int64)
    stack[:free] = pages[:free]
    return dict(lens=_i32(lens), new=_i32(new), held=_i32(held), tables=_i32(tables),
                free_pages=_i32(stack), free_count=_i32([free]), page=P,
                most=max(1, int(new.sum())))


def _plain_pages(s):
    P, T = s["page"], s["most"]
    lens, new, held = (s[k].long() for k in ("lens", "new", "held"))
    tables, stack, n = s["tables"].clone(), s["free_pages"].clone(), s["free_count"].long()
    B, W = tables.shape
    dev = tables.device
    need = (lens + new + P - 1) // P
    back, ask = (held - need).clamp(min=0), (need - held).clamp(min=0)
    back_at, ask_at = back.cumsum(0) - back, ask.cumsum(0) - ask
    col = torch.arange(W, device=dev)
    # pages given back go on top of the stack, in the order of requests and columns
    gives = (col >= need[:, None]) & (col < held[:, None])
    at = torch.where(gives, n + back_at[:, None] + col - need[:, None], len(stack))
    stack = torch.cat([stack, stack.new_zeros(1)]).scatter_(0, at.view(-1), tables.view(-1))[:-1]
    top = n + back.sum()
    # pages asked for are taken from the top, in the same order, while they last
    served = (ask == 0) | (ask_at + ask <= top)
    takes = served[:, None] & (col >= held[:, None]) & (col < need[:, None])
    from_ = (top - 1 - ask_at[:, None] - (col - held[:, None])).clamp(0, len(stack) - 1)
    tables = torch.where(takes, stack[from_], tables)
    cu = torch.cat([new.new_zeros(1), new.cumsum(0)])
    t = torch.arange(T, device=dev)
    b = torch.searchsorted(cu[1:], t, right=True)
    inside = b < B
    b = b.clamp(max=B - 1)
    pos = lens[b] + t - cu[b]
    page = tables[b, (pos // P).clamp(max=W - 1)].long()
    slot = torch.where(inside & served[b], page * P + pos % P, -1)
    return {"slots": slot, "positions": torch.where(inside, pos, -1).int(),
            "owner": torch.where(inside, b, -1).int(), "cu": cu.int(),
            "kv_len": torch.where(served, lens + new, lens).int(),
            "held": torch.where(served, need, held).int(),
            "free_count": (top - (ask * served).sum()).int(), "served": served.int(),
            "tables": tables, "free_pages": stack}


def _own_pages(s):
    import sampling_ssd_verify_gb300 as ssd

    o = ssd.page_plan(s["lens"], s["new"], s["held"], s["tables"], s["free_pages"],
                      s["free_count"], s["page"], s["most"], out=s["out"])
    return dict(o, tables=s["tables"], free_pages=s["free_pages"])


def _exact_pages(s):
    """Request by request, with a Python list for the stack."""
    P, T = s["page"], s["most"]
    lens, new, held = (s[k].tolist() for k in ("lens", "new", "held"))
    tables, room = s["tables"].tolist(), len(s["free_pages"])
    rest = s["free_pages"].tolist()
    stack = rest[:int(s["free_count"])]
    o = dict(slots=[], positions=[], owner=[], cu=[0], kv_len=[], held=[], served=[])
    for b, (l, k, h) in enumerate(zip(lens, new, held)):
        stack += tables[b][math.ceil((l + k) / P):h]
    pushed = stack + rest[len(stack):]
    gone = False
    for b, (l, k, h) in enumerate(zip(lens, new, held)):
        need = math.ceil((l + k) / P)
        gone = gone or need - h > len(stack)
        ok = need <= h or not gone
        for c in range(h, need if ok else h):
            tables[b][c] = stack.pop()
        for p in range(l, l + k):
            o["slots"].append(tables[b][p // P] * P + p % P if ok else -1)
            o["positions"].append(p)
            o["owner"].append(b)
        o["cu"].append(o["cu"][-1] + k)
        o["kv_len"].append(l + k if ok else l)
        o["held"].append(need if ok else h)
        o["served"].append(int(ok))
    for k in ("slots", "positions", "owner"):
        o[k] += [-1] * (T - len(o[k]))
    o = {k: torch.tensor(v, dtype=torch.int64) for k, v in o.items()}
    return dict(o, free_count=torch.tensor([len(stack)]), tables=torch.tensor(tables),
                free_pages=torch.tensor(pushed[:room], dtype=torch.int64))


# ---- attention: queries of all branches, and the paged cache that they read -------------------


def _prepare_attn(case, seed):
    rng = np.random.default_rng(seed)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    G, P, Hq, Hkv, D = (case[k] for k in ("G", "page", "Hq", "Hkv", "D"))
    n = rng.permutation(_even(case["n_lo"], case["n_hi"], G))
    off = np.concatenate([[0], n.cumsum()])
    R = int(off[-1])
    pre = rng.permutation(_even(case["pre_lo"], case["pre_hi"], G))
    suf = rng.permutation(_even(case["suf_lo"], case["suf_hi"], R))
    pre_pages, suf_pages = -(-pre // P), -(-suf // P)
    ids = rng.permutation(int(pre_pages.sum() + suf_pages.sum()) + 3)

    def table(count, ids):
        t = np.zeros((len(count), max(1, int(count.max()))), dtype=np.int64)
        t[np.arange(t.shape[1]) < count[:, None]] = ids
        return _i32(t)

    dt = DTYPES[case["dtype"]]
    shape = (len(ids), P, Hkv, D)
    q = torch.randn((R, Hq, D), generator=gen, device="cuda").to(dt)
    k = torch.empty(shape, dtype=dt, device="cuda").normal_(generator=gen)
    v = torch.empty(shape, dtype=dt, device="cuda").normal_(generator=gen)
    return dict(q=q, k=k, v=v, prefix_tables=table(pre_pages, ids[:pre_pages.sum()]),
                prefix_len=_i32(pre), group_off=_i32(off),
                tables=table(suf_pages, ids[pre_pages.sum():-3]), lens=_i32(suf),
                n_max=int(n.max()), pre_max=int(pre.max()), suf_max=int(suf.max()),
                scale=D ** -0.5)


def _plain_attn(s):
    q, k, v = s["q"], s["k"], s["v"]
    R, Hq, D = q.shape
    P, Hkv = k.shape[1], k.shape[2]
    G, M, dev = len(s["prefix_len"]), Hq // Hkv, q.device
    off = s["group_off"].long()
    # the rows of each group side by side, short groups filled up with row 0
    place = torch.arange(s["n_max"], device=dev)
    rows = off[:-1, None] + place
    filled = rows < off[1:, None]
    rows = torch.where(filled, rows, 0)
    x = q.float()[rows].view(G, -1, Hkv, M, D).permute(0, 2, 1, 3, 4).reshape(G, Hkv, -1, D)

    def gather(cache, tables, most):
        t = torch.arange(most, device=dev)
        return cache[tables[:, t // P].long(), t % P].permute(0, 2, 1, 3).float()

    def part(x, tables, lens, most):
        """Unnormalised sums, their weights and the largest score, over one cache's tokens."""
        ok = (torch.arange(most, device=dev) < lens[:, None])[:, None, None]
        score = x @ gather(k, tables, most).transpose(-1, -2) * s["scale"]
        score = torch.where(ok, score, -math.inf)
        top = score.amax(-1, keepdim=True) if most else torch.full_like(x[..., :1], -math.inf)
        w = torch.where(ok, torch.exp(score - torch.where(top == -math.inf, 0.0, top)), 0.0)
        return w @ gather(v, tables, most), w.sum(-1, keepdim=True), top

    def to_rows(a):
        a = a.view(G, Hkv, s["n_max"], M, -1).permute(0, 2, 1, 3, 4)
        return a[filled].reshape(R, Hkv, M, -1)

    o1, l1, m1 = (to_rows(a) for a in part(x, s["prefix_tables"], s["prefix_len"], s["pre_max"]))
    o2, l2, m2 = part(q.float().view(R, Hkv, M, D), s["tables"], s["lens"], s["suf_max"])
    m = torch.maximum(m1, m2)
    m0 = torch.where(m == -math.inf, 0.0, m)
    a1, a2 = torch.exp(m1 - m0), torch.exp(m2 - m0)
    l = l1 * a1 + l2 * a2
    out = (o1 * a1 + o2 * a2) / torch.where(l > 0, l, 1.0)
    return {"out": out.view(R, Hq, D).to(q.dtype), "lse": (m + torch.log(l)).view(R, Hq)}


def _own_attn(s):
    import sampling_ssd_verify_gb300 as ssd

    o = ssd.prefix_attention(s["q"], s["k"], s["v"], s["prefix_tables"], s["prefix_len"],
                             s["group_off"], s["tables"], s["lens"], scale=s["scale"],
                             out=s["out"])
    return {"out": o["out"], "lse": o["lse"]}


def _exact_attn(s):
    """Group by group over the keys of its prefix, then row by row over its own, in float64."""
    R, Hq, D = s["q"].shape
    P, Hkv = s["k"].shape[1:3]
    M = Hq // Hkv
    out = torch.zeros((R, Hq, D), dtype=torch.float64, device="cuda")
    lse = torch.full((R, Hq), -math.inf, dtype=torch.float64, device="cuda")
    off, pre, suf = s["group_off"].tolist(), s["prefix_len"].tolist(), s["lens"].tolist()

    def tokens(cache, table, n):
        return cache[table[:-(-n // P)].long()].reshape(-1, Hkv, D)[:n].double()

    for g, n in enumerate(pre):
        a, e = off[g], off[g + 1]
        x = s["q"][a:e].double().view(e - a, Hkv, M, D)
        kg, vg = tokens(s["k"], s["prefix_tables"][g], n), tokens(s["v"], s["prefix_tables"][g], n)
        first = torch.einsum("rhmd,thd->rhmt", x, kg) * s["scale"]
        for r in range(a, e):
            t = s["tables"][r]
            sc = torch.cat([first[r - a], torch.einsum("hmd,thd->hmt", x[r - a], tokens(s["k"], t, suf[r])) * s["scale"]], -1)
            if sc.shape[-1] == 0:
                continue
            p = torch.softmax(sc, -1)
            o = torch.einsum("hmt,thd->hmd", p[..., :n], vg) + torch.einsum("hmt,thd->hmd", p[..., n:], tokens(s["v"], t, suf[r]))
            out[r], lse[r] = o.reshape(Hq, D), torch.logsumexp(sc, -1).reshape(Hq)
    return {"out": out, "lse": lse}


# ---- what the tools call ----------------------------------------------------------------------


def prepare(case, seed):
    """The inputs, and `out`: where a program that calls again and again keeps the outputs."""
    op = case["op"]
    make = {"logits": _prepare_logits, "pages": _prepare_pages, "attn": _prepare_attn}[op]
    return dict(make(case, seed), op=op, out={})


def run(state):
    op = state["op"]
    if op == "logits":
        return _own_logits(state) if own else _plain_logits(state)
    if op == "pages":
        return _own_pages(state) if own else _plain_pages(state)
    return _own_attn(state) if own else _plain_attn(state)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "logits":
        return _exact_logits(s)
    if case["op"] == "pages":
        return _exact_pages(s)
    return _exact_attn(s)


def work(case):
    if case["op"] == "logits":
        B, N, V, es = case["B"], case["N"], case["V"], BYTES[case["dtype"]]
        b = 2 * B * N * V * es + 4 * B * (case["history"] * 3 // 4 + N + 5) + 8 * B * case["biases"]
        if case["grammar"]:
            b += B * N * ((V + 31) // 32 * 4 + 4)
        # a comparison, a product and three additions for the tokens that a penalty reaches
        return {"bytes": b, "flops": 5 * B * N * min(V, case["history"] * 3 // 4)}
    if case["op"] == "pages":
        B = case["B"]
        T = int(_even(case["new_lo"], case["new_hi"], B).sum())
        # lengths in and out, a slot, a position and an owner for each token, the pages that move
        return {"bytes": 4 * (7 * B + 2) + 16 * T + 8 * (T // case["page"]), "flops": 10 * T}
    G, Hq, Hkv, D = case["G"], case["Hq"], case["Hkv"], case["D"]
    n = _even(case["n_lo"], case["n_hi"], G)
    R = int(n.sum())
    pre = int(_even(case["pre_lo"], case["pre_hi"], G).sum())
    suf = int(_even(case["suf_lo"], case["suf_hi"], R).sum())
    b = 2 * (2 * R * Hq * D + 2 * (pre + suf) * Hkv * D) + 4 * R * Hq
    b += 4 * ((pre + suf) // case["page"] + 2 * G + R)
    return {"bytes": b, "flops": 4 * Hq * D * (pre / G * R + suf)}
