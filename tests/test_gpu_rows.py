"""append_path and fork_rows against row-by-row loops: what they move is compared bit for bit."""

import numpy as np
import pytest

import sampling_ssd_verify_gb300 as ssd
from tests.parity import i32, torch_dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    ssd.build()
    ssd.lib()


def filled(shape, dtype, gen):
    """Bytes of any kind: a copy keeps them whatever they mean."""
    torch, dev = torch_dev()
    es = torch.empty(0, dtype=dtype).element_size()
    x = torch.randint(0, 256, (*shape[:-1], shape[-1] * es), generator=gen, device=dev,
                      dtype=torch.uint8)
    return x.view(dtype)


def raw(t):
    import torch
    return t.contiguous().view(torch.uint8)


LAYOUT = {"nhd": (0, 1, 2, 3, 4), "hnd": (0, 1, 3, 2, 4), "last": (1, 2, 0, 3, 4)}


def laid_out(x, order):
    """The same [L, X, Y, H, D] values with another order in memory."""
    perm = LAYOUT[order]
    back = [perm.index(i) for i in range(5)]
    return x.permute(perm).contiguous().permute(back)


# ---- append_path ---------------------------------------------------------------------------
def append_case(B, N, L, H, D, page, dtype, seed=0, chain=False, order="nhd", pad=3):
    torch, dev = torch_dev()
    rng = np.random.default_rng(seed)
    gen = torch.Generator(device=dev).manual_seed(seed)
    depth = N - 1
    new = rng.integers(0, N + 1, B)
    path = np.full((B, max(1, depth)), -1)
    for b in range(B):
        n = max(0, new[b] - 1)
        path[b, :n] = np.sort(rng.choice(np.arange(1, N), n, replace=False)) if n else []
    lens = rng.integers(0, 3 * page, B)
    pages = -(-(lens + new) // page)
    ids = rng.permutation(int(pages.sum()) + 2)
    cu = np.concatenate([[0], np.cumsum(new)])
    T = int(cu[-1])
    slots, owner = np.full(T + pad, -1, dtype=np.int64), np.full(T + pad, -1)
    at = np.concatenate([[0], np.cumsum(pages)])
    for b in range(B):
        for i in range(new[b]):
            pos = lens[b] + i
            slots[cu[b] + i] = ids[at[b] + pos // page] * page + pos % page
            owner[cu[b] + i] = b
    if T:
        slots[rng.integers(0, T)] = -1   # one of a request that got no pages
    s = dict(slots=torch.from_numpy(slots).to(dev), owner=i32(owner), cu=i32(cu),
             path=None if chain else i32(path))
    for name in ("k", "v"):
        s[name] = laid_out(filled((L, B, N, H, D), dtype, gen), order)
        s[name + "_cache"] = laid_out(filled((L, len(ids), page, H, D), dtype, gen), order)
    return s


def appended(s):
    """The caches afterwards, token by token."""
    P = s["k_cache"].shape[2]
    out = {}
    slots, owner, cu = (s[n].tolist() for n in ("slots", "owner", "cu"))
    for name in ("k", "v"):
        c = s[name + "_cache"].clone()
        for t, slot in enumerate(slots):
            if slot < 0:
                continue
            b = owner[t]
            i = t - cu[b]
            node = i if s["path"] is None or i == 0 else int(s["path"][b, i - 1])
            c[:, slot // P, slot % P] = s[name][:, b, node]
        out[name + "_cache"] = c
    return out


def run_append(s, **kw):
    return ssd.append_path(s["k"], s["v"], s["k_cache"], s["v_cache"], s["slots"], s["owner"],
                           s["cu"], s["path"], **kw)


@pytest.mark.parametrize("dt", ["bfloat16", "float32", "uint8"])
@pytest.mark.parametrize("B,N,L,H,D,page", [
    (1, 1, 1, 1, 16, 1), (1, 5, 32, 8, 128, 16), (3, 2, 5, 3, 80, 5), (40, 9, 3, 2, 64, 20),
    (300, 4, 2, 1, 16, 64), (7, 64, 2, 4, 256, 16), (2, 3, 70, 1, 48, 8),
])
@pytest.mark.parametrize("order", ["nhd", "hnd", "last"])
@pytest.mark.parametrize("chain", [False, True])
def test_append(dt, B, N, L, H, D, page, order, chain):
    torch, dev = torch_dev()
    s = append_case(B, N, L, H, D, page, getattr(torch, dt), seed=B + N, chain=chain, order=order)
    want = appended(s)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    assert run_append(s, dev_status=status) is None
    for name, c in want.items():
        assert torch.equal(raw(s[name]), raw(c)), name
    assert int(status.item()) == 0


def test_append_of_one_layer_and_of_keys_alone():
    torch, dev = torch_dev()
    s = append_case(5, 4, 1, 2, 64, 16, torch.bfloat16)
    want = appended(s)
    ssd.append_path(s["k"][0], s["v"][0], s["k_cache"][0], s["v_cache"][0], s["slots"], s["owner"],
                    s["cu"], s["path"])
    assert torch.equal(raw(s["k_cache"]), raw(want["k_cache"]))
    assert torch.equal(raw(s["v_cache"]), raw(want["v_cache"]))
    s = append_case(5, 4, 3, 1, 576, 16, torch.bfloat16)
    want, before = appended(s), s["v_cache"].clone()
    ssd.append_path(s["k"], None, s["k_cache"], None, s["slots"], s["owner"], s["cu"], s["path"])
    assert torch.equal(raw(s["k_cache"]), raw(want["k_cache"]))
    assert torch.equal(raw(s["v_cache"]), raw(before))


@pytest.mark.parametrize("orders", [("nhd", "hnd", "last", "nhd"), ("hnd", "nhd", "nhd", "last"),
                                    ("last", "hnd", "hnd", "nhd")])
@pytest.mark.parametrize("B,L", [(3, 2), (200, 40)])
def test_append_with_a_layout_each(orders, B, L):
    """Keys, values and both caches have strides of their own."""
    torch, dev = torch_dev()
    s = append_case(B, 6, L, 5, 64, 16, torch.bfloat16, seed=B)
    want = appended(s)
    for name, order in zip(("k", "v", "k_cache", "v_cache"), orders):
        s[name] = laid_out(s[name], order)
    run_append(s)
    assert torch.equal(raw(s["k_cache"]), raw(want["k_cache"]))
    assert torch.equal(raw(s["v_cache"]), raw(want["v_cache"]))


def test_append_with_views_of_larger_tensors():
    """Nodes that are pieces of a projection, caches that are pieces of a pool."""
    torch, dev = torch_dev()
    s = append_case(6, 5, 2, 2, 64, 16, torch.bfloat16)
    want = appended(s)
    qkv = torch.zeros((2, 6, 5, 9, 64), dtype=torch.bfloat16, device=dev)
    pool = torch.zeros((2, *s["k_cache"].shape), dtype=torch.bfloat16, device=dev)
    pool = pool.permute(1, 2, 0, 3, 4, 5).contiguous().permute(2, 0, 1, 3, 4, 5)
    views = dict(k=qkv[..., 5:7, :], v=qkv[..., 7:9, :], k_cache=pool[0], v_cache=pool[1])
    for n, x in views.items():
        x.copy_(s[n])
    run_append(dict(s, **views))
    assert torch.equal(raw(pool[0]), raw(want["k_cache"]))
    assert torch.equal(raw(pool[1]), raw(want["v_cache"]))


def test_append_passes_over_what_is_out_of_range():
    torch, dev = torch_dev()
    status = torch.zeros(1, dtype=torch.int32, device=dev)

    def flags(bit, **kw):
        s = append_case(6, 5, 2, 2, 64, 16, torch.bfloat16, seed=3)
        slots = s["slots"].clone()
        t = int((slots >= 0).nonzero()[-1])   # the last token that is stored
        b = int(s["owner"][t])
        for name, x in kw.items():
            x = x(s, t, b)
            if name == "path":
                i = t - int(s["cu"][b])
                assert i > 0
                s["path"][b, i - 1] = x
            else:
                s[name][t if name != "cu" else b] = x
        good = dict(s, slots=slots.clone())
        lost = [t] if "cu" not in kw else [i for i in range(t + 1) if int(s["owner"][i]) == b]
        good["slots"][lost] = -1
        want = appended(good)
        status.zero_()
        run_append(s, dev_status=status)
        assert int(status.item()) == bit
        for name, c in want.items():
            assert torch.equal(raw(s[name]), raw(c))

    pages = append_case(6, 5, 2, 2, 64, 16, torch.bfloat16, seed=3)["k_cache"].shape[1]
    for slot in (pages * 16, 2 ** 62):
        flags(ssd.DEV_BAD_PAGE, slots=lambda s, t, b: slot)
    for owner in (-1, 6, 2 ** 31 - 1, -2 ** 31):
        flags(ssd.DEV_BAD_LENGTH, owner=lambda s, t, b: owner)
    for node in (-1, 5, 2 ** 31 - 1):
        flags(ssd.DEV_BAD_LENGTH, path=lambda s, t, b: node)
    for first in (2 ** 31 - 1, -2 ** 31, -100):
        flags(ssd.DEV_BAD_LENGTH, cu=lambda s, t, b: first)


def test_append_on_streams_in_graphs_and_of_nothing():
    torch, dev = torch_dev()
    s = append_case(9, 6, 4, 2, 128, 16, torch.float16)
    want = appended(s)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    run_append(s, stream=st)
    st.synchronize()
    assert torch.equal(raw(s["k_cache"]), raw(want["k_cache"]))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run_append(s)
    s["k"].copy_(s["v"])
    g.replay()
    assert torch.equal(raw(s["k_cache"][:, 0]), raw(appended(s)["k_cache"][:, 0]))
    assert torch.equal(raw(s["k_cache"]), raw(appended(s)["k_cache"]))
    before = s["k_cache"].clone()
    run_append(dict(s, slots=s["slots"][:0], owner=s["owner"][:0]))
    assert torch.equal(raw(s["k_cache"]), raw(before))


# ---- fork_rows -----------------------------------------------------------------------------
def fork_case(S, B, W, page, free, L=0, H=2, D=16, dtype="bfloat16", seed=0, src=None,
              shared=True, order="nhd", spare=1, cap=None):
    torch, dev = torch_dev()
    rng = np.random.default_rng(seed)
    gen = torch.Generator(device=dev).manual_seed(seed)
    lens = rng.integers(0, (W - spare) * page + 1, S)
    held = np.minimum(W, -(-lens // page) + rng.integers(0, spare + 1, S))
    table = np.full((S, W), -77)
    shares, at = [], 0
    for r in range(S):
        c = 0
        if r and shared and rng.random() < 0.5:   # full pages of both rows
            o = int(rng.integers(0, r))
            c = int(min(lens[r] // page, lens[o] // page))
            table[r, :c] = table[o, :c]
            for p in table[r, :c]:
                shares[p] += 1
        n = int(held[r]) - c
        table[r, c:c + n] = np.arange(at, at + n)
        shares += [0] * n
        at += n
    total = at + free + 2
    ids = rng.permutation(total)
    used = table >= 0
    table[used] = ids[table[used]]
    share = np.zeros(total, dtype=int)
    share[ids[:at]] = shares
    room = total if cap is None else cap
    stack = np.full(room, -9)
    stack[:free] = ids[at:at + free]
    if src is None:
        src = rng.integers(-1, S, B)
    s = dict(src=np.asarray(src), lens=lens, held=held, tables=table, shares=share, free_pages=stack,
             free_count=np.array([free]), page=page)
    for name in ("k_cache", "v_cache"):
        s[name] = laid_out(filled((L, total, page, H, D), getattr(torch, dtype), gen), order) \
            if L else None
    return s


def forked(s):
    """Everything afterwards, row by row; the device status too."""
    P, W = s["page"], s["tables"].shape[1]
    n, cap = int(s["free_count"][0]), len(s["free_pages"])
    flags = 0
    stack = s["free_pages"][:n].tolist()
    holders = (s["shares"] + 1).tolist()
    src, S = s["src"].tolist(), len(s["lens"])
    goes_on = set(src)
    for r in range(S):
        if r not in goes_on:
            for p in s["tables"][r, :s["held"][r]].tolist():
                holders[p] -= 1
                if holders[p] == 0:
                    stack.append(p)
    pushed = (stack + s["free_pages"].tolist()[len(stack):])[:cap]
    o = dict(tables=np.full((len(src), W), -1), lens=[], held=[], served=[])
    caches = {c: None if s[c] is None else s[c].clone() for c in ("k_cache", "v_cache")}
    seen, empty = set(), False
    for b, r in enumerate(src):
        pages, length, ok = [], 0, 1
        if r >= 0 and r not in seen:
            seen.add(r)
            pages, length = s["tables"][r, :s["held"][r]].tolist(), s["lens"][r]
        elif r >= 0:
            full, tail = divmod(int(s["lens"][r]), P)
            empty = empty or (tail > 0 and not stack)
            if tail and empty:
                ok = 0
                flags |= ssd.DEV_NO_PAGES
            else:
                pages, length = s["tables"][r, :full].tolist(), s["lens"][r]
                for p in pages:
                    holders[p] += 1
                if tail:
                    p = stack.pop()
                    holders[p] = 1
                    for c in caches.values():
                        if c is not None:
                            c[:, p, :tail] = c[:, int(s["tables"][r, full]), :tail]
                    pages.append(p)
        o["tables"][b, :len(pages)] = pages
        o["lens"].append(int(length))
        o["held"].append(len(pages))
        o["served"].append(ok)
    if len(stack) > cap:
        flags |= ssd.DEV_BAD_LENGTH
    o.update(shares=[max(0, h - 1) for h in holders], free_count=[min(len(stack), cap)],
             free_pages=pushed, **caches)
    return o, flags


INPUTS = ("src", "lens", "held", "tables", "shares", "free_pages", "free_count")


def on_gpu(s):
    return {k: i32(v) if k in INPUTS else v for k, v in s.items()}


def run_fork(d, **kw):
    return ssd.fork_rows(d["src"], d["lens"], d["held"], d["tables"], d["shares"], d["free_pages"],
                         d["free_count"], d["page"], d["k_cache"], d["v_cache"], **kw)


def check_fork(s, **kw):
    torch, dev = torch_dev()
    want, flags = forked(s)
    d = on_gpu(s)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    for _ in range(2):                   # the same inputs again give the same results
        status.zero_()
        o = run_fork(d, dev_status=status, **kw)
        for name in ("tables", "lens", "held", "served", "shares", "free_count"):
            np.testing.assert_array_equal(o[name].cpu().numpy(), np.asarray(want[name]), name)
        np.testing.assert_array_equal(d["free_pages"].cpu().numpy(), np.asarray(want["free_pages"]))
        for name in ("k_cache", "v_cache"):
            if s[name] is not None:
                assert torch.equal(raw(d[name]), raw(want[name]))
        assert int(status.item()) == flags
    for name in ("src", "lens", "held", "tables", "shares", "free_count"):
        np.testing.assert_array_equal(d[name].cpu().numpy(), np.asarray(s[name]))
    return o


@pytest.mark.parametrize("S,B,W,page,free", [
    (1, 1, 1, 1, 0), (1, 8, 94, 16, 8), (4, 4, 3, 16, 20), (5, 12, 40, 5, 3), (64, 64, 70, 16, 80),
    (300, 300, 33, 64, 40), (1500, 40, 10, 8, 50), (30, 2000, 50, 20, 2000), (8192, 8192, 3, 16, 99),
    (700, 700, 200, 4, 300),
])
def test_fork(S, B, W, page, free):
    for seed in range(3):
        check_fork(fork_case(S, B, W, page, free, seed=seed, spare=min(1, W - 1)))


@pytest.mark.parametrize("dt,H,D", [("bfloat16", 8, 128), ("float32", 3, 20), ("uint8", 1, 16),
                                    ("float16", 5, 64)])
@pytest.mark.parametrize("order", ["nhd", "hnd", "last"])
@pytest.mark.parametrize("page,L", [(16, 3), (1, 2), (20, 1), (128, 2)])
def test_fork_copies_last_pages(dt, H, D, order, page, L):
    check_fork(fork_case(9, 40, 4, page, 60, L=L, H=H, D=D, dtype=dt, order=order, seed=page))


@pytest.mark.parametrize("src", [
    [-1, -1, -1], [0, 1, 2], [2, 1, 0], [1, 1, 1], [2, -1, 2], [0], [1, 1, 1, 1, 1, 1, 1, 1, 1, 1],
])
@pytest.mark.parametrize("free", [0, 1, 20])
def test_fork_of_few_rows(src, free):
    check_fork(fork_case(3, len(src), 9, 4, free, L=2, src=src, seed=free))
    check_fork(fork_case(3, len(src), 9, 4, free, L=2, src=src, seed=free, shared=False))


def test_fork_gives_back_pages_that_the_same_call_takes():
    """The stack passes the array's end in between; what stays past it is lost, and flagged."""
    for cap in (0, 1, 3, 7, 40):
        src = [1, 1, 1, 1, 1]
        check_fork(fork_case(4, 5, 6, 8, min(cap, 1), src=src, shared=False, cap=cap, seed=cap, L=1))


def test_fork_of_keys_alone_and_of_one_layer():
    torch, dev = torch_dev()
    s = fork_case(6, 9, 5, 16, 20, L=1, H=1, D=576)
    want, _ = forked(s)
    d = on_gpu(s)
    before = s["v_cache"].clone()
    o = run_fork(dict(d, k_cache=s["k_cache"][0], v_cache=None))
    assert torch.equal(raw(s["k_cache"]), raw(want["k_cache"]))
    assert torch.equal(raw(s["v_cache"]), raw(before))
    np.testing.assert_array_equal(o["tables"].cpu().numpy(), want["tables"])


def test_fork_with_a_layout_each_and_tables_in_wider_rows():
    torch, dev = torch_dev()
    for orders in (("nhd", "hnd"), ("hnd", "last"), ("last", "nhd")):
        s = fork_case(40, 60, 6, 16, 50, L=3, H=3, D=32, seed=4)
        want, _ = forked(s)
        d = on_gpu(s)
        wide = torch.full((40, 19), -5, dtype=torch.int32, device=dev)
        wide[:, 7:13] = d["tables"]
        d.update(tables=wide[:, 7:13], k_cache=laid_out(s["k_cache"], orders[0]),
                 v_cache=laid_out(s["v_cache"], orders[1]))
        o = run_fork(d)
        np.testing.assert_array_equal(o["tables"].cpu().numpy(), want["tables"])
        np.testing.assert_array_equal(o["shares"].cpu().numpy(), want["shares"])
        for name in ("k_cache", "v_cache"):
            assert torch.equal(raw(d[name]), raw(want[name]))
        assert bool((wide[:, :7] == -5).all()) and bool((wide[:, 13:] == -5).all())


def test_fork_of_tables_of_many_pages():
    """More pages than a warp has in flight, over one CTA and over a cluster."""
    check_fork(fork_case(3, 2, 900, 1, 5, src=[1, 1], seed=2, shared=False))
    check_fork(fork_case(3, 2, 30000, 1, 5, src=[2, 2], seed=3))


def test_fork_chained_on_streams_and_in_a_graph():
    """The outputs of a call are the inputs of the next."""
    torch, dev = torch_dev()
    rng = np.random.default_rng(5)
    s = fork_case(12, 12, 9, 8, 60, L=2, seed=5)
    d, out = on_gpu(s), [{}, {}]
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    for i in range(6):
        want, _ = forked(s)
        o = run_fork(d, out=out[i % 2], stream=st)
        st.synchronize()
        for name in ("tables", "lens", "held", "served", "shares", "free_count"):
            np.testing.assert_array_equal(o[name].cpu().numpy(), np.asarray(want[name]), name)
        for name in ("k_cache", "v_cache"):
            assert torch.equal(raw(d[name]), raw(want[name]))
        src = rng.integers(-1, 12, 12)
        s = dict(s, src=src, **{n: np.asarray(want[n]) for n in INPUTS if n != "src"},
                 k_cache=d["k_cache"], v_cache=d["v_cache"])
        d = dict(d, src=i32(src), **{n: o[n] for n in ("tables", "lens", "held", "shares",
                                                       "free_count")})
    want, _ = forked(s)
    keep = {}
    run_fork(d, out=keep)
    for name in ("tables", "shares"):
        keep[name].zero_()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run_fork(d, out=keep)
    for _ in range(2):
        g.replay()
    for name in ("tables", "lens", "held", "served", "shares", "free_count"):
        np.testing.assert_array_equal(keep[name].cpu().numpy(), np.asarray(want[name]), name)


def test_fork_of_rows_that_are_inconsistent():
    torch, dev = torch_dev()
    status = torch.zeros(1, dtype=torch.int32, device=dev)

    def call(bit, src, rows, L=0, **kw):
        s = fork_case(5, len(src), 6, 8, 9, src=src, shared=False, seed=1)
        s["lens"][:] = 13
        s["held"][:] = 2
        s["tables"][:, :2] = np.arange(10).reshape(5, 2)
        s["free_pages"][:9] = np.arange(10, 19)
        s["shares"] = np.zeros(40, dtype=int)
        for name, (at, x) in kw.items():
            s[name][at] = x
        for name in ("k_cache", "v_cache"):
            s[name] = torch.ones((L, 40, 8, 1, 16), device=dev) if L else None
        d = on_gpu(s)
        status.zero_()
        o = {k: v.cpu().numpy() for k, v in run_fork(d, dev_status=status).items()}
        assert int(status.item()) == bit
        for b, r in enumerate(rows):
            assert o["tables"][b].tolist() == r + [-1] * (6 - len(r)), b
            assert o["held"][b] == len(r)
        return o, d["free_pages"].cpu().numpy()

    BAD, PAGE = ssd.DEV_BAD_LENGTH, ssd.DEV_BAD_PAGE
    good = [[0, 1], [0, 9]]            # rows 2 to 4 end, and 9 is the last page given back
    for name, x in (("lens", -1), ("lens", 17), ("held", -1), ("held", 7), ("held", 1)):
        o, stack = call(BAD, [0, 0, 1, 1], good + [[], []], **{name: (1, x)})
        assert o["served"].tolist() == [1, 1, 0, 0] and o["lens"].tolist() == [13, 13, 0, 0]
        o, stack = call(BAD, [0, 0], good, **{name: (1, x)})
        assert stack[9:15].tolist() == [4, 5, 6, 7, 8, 9] and o["free_count"][0] == 14
    for x in (-2, 5, 2 ** 31 - 1, -2 ** 31):
        o, _ = call(BAD, [0, 1, x, 3, 4, 0], [[0, 1], [2, 3], [], [6, 7], [8, 9], [0, 5]])
        assert o["served"].tolist() == [1, 1, 0, 1, 1, 1]
    for x in (-1, 10 ** 6):
        o, stack = call(BAD, [0, 1, 2, 3, 4], [[0, 1], [2, 3], [4, 5], [6, 7], [8, 9]],
                    free_count=(0, x))
        assert o["free_count"][0] == (0 if x < 0 else len(stack))
    for x in (-1, 40, 2 ** 31 - 1):
        # given back; shared; the last page of a fork
        o, _ = call(PAGE, [1, 2, 3, 4], [[2, 3], [4, 5], [6, 7], [8, 9]], tables=((0, 1), x))
        assert o["free_count"][0] == 10
        o, _ = call(PAGE, [0, 0, 1, 2, 3, 4], [[x, 1], [x, 18]] + [[2, 3], [4, 5], [6, 7], [8, 9]],
                    tables=((0, 0), x))
        assert o["shares"].sum() == 0
        o, _ = call(0, [0, 0, 1, 2, 3, 4], [[0, x], [0, 18]] + [[2, 3], [4, 5], [6, 7], [8, 9]],
                    tables=((0, 1), x))
        assert o["shares"].sum() == 1
        call(PAGE, [0, 0, 1, 2, 3, 4], [[0, x], [0, 18]] + [[2, 3], [4, 5], [6, 7], [8, 9]], L=3,
             tables=((0, 1), x))         # its tokens are not there to be copied
    # a page given back more often than it is held
    o, stack = call(PAGE, [2, 3, 4], [[4, 5], [6, 7], [8, 9]], tables=((1, 0), 0))
    assert stack[9:12].tolist() == [1, 0, 3] and o["free_count"][0] == 12


def test_refusals():
    torch, dev = torch_dev()
    s = on_gpu(fork_case(4, 5, 6, 8, 9, L=2))
    run_fork(s)
    k = s["k_cache"]
    for kw in (dict(src=s["src"].long()), dict(lens=s["lens"][:3]), dict(held=s["held"][:3]),
               dict(tables=s["tables"][:3]), dict(tables=s["tables"].t().contiguous().t()),
               dict(shares=s["shares"].long()), dict(free_count=s["free_count"].repeat(2)),
               dict(src=s["src"].cpu()), dict(k_cache=k[:, :-1]), dict(k_cache=None),
               dict(v_cache=k.half()), dict(page=4), dict(k_cache=k[..., :4], v_cache=None),
               dict(v_cache=k), dict(shares=s["shares"][:3]), dict(tables=s["tables"][:, :0])):
        with pytest.raises(ssd.SSDError):
            run_fork(dict(s, **kw))
    for name in ("tables", "lens", "held", "shares", "free_count"):
        if s[name].shape == (5,) or name in ("shares", "free_count"):
            with pytest.raises(ssd.SSDError):
                run_fork(s, out={name: s[name]})
    with pytest.raises(ssd.SSDError):
        run_fork(s, workspace=torch.empty(256, dtype=torch.uint8, device=dev))
    a = append_case(4, 3, 2, 2, 64, 16, torch.bfloat16)
    run_append(a)
    for kw in (dict(k=a["k"][:1], v=a["v"][:1]), dict(k=a["k"].half(), v=a["v"].half()),
               dict(v=None), dict(v_cache=None), dict(slots=a["slots"].int()),
               dict(owner=a["owner"][:-1]), dict(cu=a["cu"][:-1]), dict(path=a["path"].long()),
               dict(k=a["k"].transpose(3, 4), v=a["v"].transpose(3, 4)),
               dict(v_cache=a["k_cache"]), dict(k=a["k_cache"], v=a["v_cache"]),
               dict(k=a["k"].cpu()), dict(k_cache=a["k_cache"].cpu()),
               dict(k=a["k"][..., :4], v=a["v"][..., :4], k_cache=a["k_cache"][..., :4],
                    v_cache=a["v_cache"][..., :4])):
        with pytest.raises(ssd.SSDError):
            run_append(dict(a, **kw))


@pytest.mark.parametrize("page", [2 ** 31, 2 ** 40, -2 ** 40])
def test_page_sizes_beyond_32_bits_are_refused(page):
    s = on_gpu(fork_case(4, 5, 6, 8, 9, L=2))
    with pytest.raises(ssd.SSDError):
        run_fork(dict(s, page=page, k_cache=None, v_cache=None))


def test_append_with_a_path_of_no_columns():
    """Only node 0 has a place; rows past it are passed over and flagged, as with a path that is
    too short."""
    torch, dev = torch_dev()
    gen = torch.Generator(device=dev).manual_seed(0)
    k, c = filled((2, 3, 4, 2, 64), torch.bfloat16, gen), filled((2, 9, 16, 2, 64), torch.bfloat16, gen)
    slots = torch.tensor([5, 20, 21, 40, -1], device=dev)
    owner, cu = i32([0, 1, 1, 2, -1]), i32([0, 1, 3, 4])
    for path in (torch.empty((3, 0), dtype=torch.int32, device=dev), i32([[1], [2], [3]])[:, :0]):
        cache, status = c.clone(), torch.zeros(1, dtype=torch.int32, device=dev)
        ssd.append_path(k, None, cache, None, slots, owner, cu, path, dev_status=status)
        want = c.clone()
        for slot, b in ((5, 0), (20, 1), (40, 2)):
            want[:, slot // 16, slot % 16] = k[:, b, 0]
        assert torch.equal(raw(cache), raw(want))
        assert int(status.item()) == ssd.DEV_BAD_LENGTH


@pytest.mark.parametrize("L", [0, 3])
@pytest.mark.parametrize("x", [-1, 40, -9, 2 ** 31 - 1, -2 ** 31])
@pytest.mark.parametrize("W", [6, 900])
def test_fork_passes_over_stack_entries_that_are_no_pages(L, x, W):
    """The row that would take one is left empty and not served, and the entry is off the stack;
    rows after it take the next."""
    torch, dev = torch_dev()
    s = fork_case(5, 5, W, 8, 9, src=[0, 0, 1, 0, 1], shared=False, seed=1)
    s["lens"][:] = 13
    s["held"][:] = 2
    s["tables"][:, :2] = np.arange(10).reshape(5, 2)
    s["free_pages"][:9] = np.arange(10, 19)
    s["shares"] = np.zeros(40, dtype=int)
    s["free_count"][0] = 2               # below the six pages that rows 2 to 4 give back
    gen = torch.Generator(device=dev).manual_seed(2)
    for name in ("k_cache", "v_cache"):
        s[name] = filled((L, 40, 8, 1, 16), torch.bfloat16, gen) if L else None

    def call(src):
        s["src"] = np.array(src)
        d = on_gpu(s)
        for name in ("k_cache", "v_cache"):
            d[name] = s[name].clone() if L else None
        status = torch.zeros(1, dtype=torch.int32, device=dev)
        o = {k: v.cpu().numpy() for k, v in run_fork(d, dev_status=status).items()}
        for k in ("tables", "lens", "held", "served", "shares"):
            o[k] = o[k].tolist()
        o["tables"] = [[p for p in r if p != -1] for r in o["tables"]]
        return o, int(status.item()), d

    # no row gives pages back: the stack alone, of which an entry is no page
    for bad, pages in ((1, (None, 10)), (0, (11, None))):
        s["free_pages"][:2] = [10, 11]
        s["free_pages"][bad] = x
        o, status, d = call([0, 1, 2, 3, 4, 0, 1])
        assert status == ssd.DEV_BAD_PAGE
        want = [[0, 1], [2, 3], [4, 5], [6, 7], [8, 9]]
        for row, page in zip((0, 2), pages):
            want.append([] if page is None else [row, page])
        assert o["tables"] == want
        assert o["served"] == [1] * 5 + [int(p is not None) for p in pages]
        assert o["held"] == [len(r) for r in want] and o["lens"] == [13 if r else 0 for r in want]
        assert sum(o["shares"]) == 1 and o["shares"][0 if pages[0] else 2] == 1
        assert o["free_count"][0] == 0
        for name in ("k_cache", "v_cache"):
            if L:
                c = s[name].clone()
                old, new = (1, pages[0]) if pages[0] else (3, pages[1])
                c[:, new, :5] = c[:, old, :5]
                assert torch.equal(raw(d[name]), raw(c))
    # pages given back are taken first: the entry below them is reached by the last row alone
    s["free_pages"][:2] = [10, x]
    o, status, d = call([0, 0, 0, 0, 0, 0, 0, 0, 0, 0])
    assert status == ssd.DEV_BAD_PAGE
    assert o["tables"] == [[0, 1]] + [[0, p] for p in (9, 8, 7, 6, 5, 4, 3, 2)] + [[]]
    assert o["served"] == [1] * 9 + [0] and o["free_count"][0] == 1 and o["shares"][0] == 8
    # and where no row takes it, it stays
    o, status, d = call([0, 0, -1])
    assert status == 0 and o["free_count"][0] == 9 and int(d["free_pages"][1]) == x
