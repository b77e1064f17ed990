"""prefix_attention against the definition in float64, row by row.

Tolerance, from the formulas.  A score is a sum of D exact products, scaled,
and lessened by a maximum, in float32: with S the largest scale * sum |q k| of
the row it is off by at most rs = (D + 4) 2^-23 S + 2^-21 (the last term: the
exponential).  A weight is rounded to the type (eps / 2) and its sums run over
n tokens in float32 (n 2^-23); with A = sum p |v| over the normalised weights
  |out - exact| <= A (eps/2 + 2 rs + (n + 8) 2^-23) + eps/2 |exact|,
and for float16, whose small weights lose steps of 2^-24, half a step of each
weight more.  |lse - exact| <= rs + n 2^-24 + 2^-21 + 2^-23 |exact|.
"""

import math

import numpy as np
import pytest

import sampling_ssd_verify_gb300 as ssd
from tests.parity import i32, torch_dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    ssd.build()
    ssd.lib()


def make(sizes, pre, suf, Hq, Hkv, D, page, dtype, seed=0, order="nhd", own=True, spread=1.0,
         spare=3):
    """Groups of `sizes` rows with `pre` tokens each, rows with `suf` own tokens."""
    torch, dev = torch_dev()
    rng = np.random.default_rng(seed)
    gen = torch.Generator(device=dev).manual_seed(seed)
    R = int(sum(sizes))
    off = np.concatenate([[0], np.cumsum(sizes)]).astype(int)
    pre, suf = np.asarray(pre), np.asarray(suf) if own else np.zeros(R, int)
    np_, ns = -(-pre // page), -(-suf // page)
    total = int(np_.sum() + ns.sum()) + spare
    ids = rng.permutation(total)

    def table(n, ids):
        # unused columns hold what is no page: they are never read
        t = np.full((len(n), max(1, int(n.max(initial=0))) + 2), -12345)
        t[np.arange(t.shape[1]) < n[:, None]] = ids
        return i32(t)

    shape = {"nhd": (total, page, Hkv, D), "hnd": (total, Hkv, page, D),
             "pnh": (page, total, Hkv, D)}[order]
    perm = {"nhd": (0, 1, 2, 3), "hnd": (0, 2, 1, 3), "pnh": (1, 0, 2, 3)}[order]
    k = (torch.randn(shape, generator=gen, device=dev) * spread).to(dtype).permute(perm)
    v = torch.randn(shape, generator=gen, device=dev).to(dtype).permute(perm)
    q = (torch.randn((R, Hq, D), generator=gen, device=dev) * spread).to(dtype)
    s = dict(q=q, k=k, v=v, pt=table(np_, ids[:np_.sum()]), pl=i32(pre), off=i32(off),
             t=table(ns, ids[np_.sum():np_.sum() + ns.sum()]) if own else None,
             l=i32(suf) if own else None)
    s["groups"] = np.repeat(np.arange(len(sizes)), sizes)
    s["pre"], s["suf"] = pre, suf
    return s


def poison(s):
    """NaN in every cache entry that no row reads."""
    torch, dev = torch_dev()
    pages, page = s["k"].shape[:2]
    used = torch.zeros((pages, page), dtype=torch.bool, device=dev)
    for tab, lens in ((s["pt"], s["pre"]), (s["t"], s["suf"])):
        if tab is None:
            continue
        for i, n in enumerate(lens):
            t = torch.arange(int(n), device=dev)
            used[tab[i][t // page].long(), t % page] = True
    for c in (s["k"], s["v"]):
        c[~used] = float("nan")


def call(s, **kw):
    return ssd.prefix_attention(s["q"], s["k"], s["v"], s["pt"], s["pl"], s["off"], s["t"], s["l"],
                                **kw)


def check(s, o, scale=None, rows=None, eps_of=None):
    torch, dev = torch_dev()
    R, Hq, D = s["q"].shape
    page, Hkv = s["k"].shape[1:3]
    M = Hq // Hkv
    scale = D ** -0.5 if scale is None else scale
    eps = torch.finfo(s["q"].dtype).eps
    half = s["q"].dtype == torch.float16
    assert o["out"].shape == (R, Hq, D) and o["out"].dtype == s["q"].dtype

    def tokens(cache, table, n):
        t = torch.arange(int(n), device=dev)
        return cache[table[t // page].long(), t % page].double()

    worst = 0.0
    for r in range(R) if rows is None else rows:
        g = s["groups"][r]
        parts = [(s["pt"][g], s["pre"][g])]
        if s["t"] is not None:
            parts.append((s["t"][r], s["suf"][r]))
        k = torch.cat([tokens(s["k"], t, n) for t, n in parts])
        v = torch.cat([tokens(s["v"], t, n) for t, n in parts])
        n = len(k)
        got, lse = o["out"][r].double(), o["lse"][r].double() if "lse" in o else None
        if n == 0:
            assert bool((got == 0).all())
            assert lse is None or bool((lse == -math.inf).all())
            continue
        x = s["q"][r].double().view(Hkv, M, D)
        sc = torch.einsum("hmd,thd->hmt", x, k) * scale
        S = (torch.einsum("hmd,thd->hmt", x.abs(), k.abs()) * abs(scale)).amax(-1, keepdim=True)
        p = torch.softmax(sc, -1)
        want = torch.einsum("hmt,thd->hmd", p, v)
        A = torch.einsum("hmt,thd->hmd", p, v.abs())
        rs = (D + 4) * 2.0 ** -23 * S + 2.0 ** -21
        tol = A * (eps / 2 + 2 * rs + (n + 8) * 2.0 ** -23) + eps / 2 * want.abs()
        if half:
            tol = tol + 2.0 ** -25 * (v.abs().sum(0)[:, None] + 1)
        err = (got.view(Hkv, M, D) - want).abs()
        assert bool((err <= tol).all()), (r, float((err / tol).max()))
        worst = max(worst, float((err / tol).max()))
        if lse is not None:
            ref = torch.logsumexp(sc, -1)
            e = (lse.view(Hkv, M) - ref).abs()
            t2 = rs[..., 0] + n * 2.0 ** -24 + 2.0 ** -21 + 2.0 ** -23 * ref.abs()
            assert bool((e <= t2).all()), (r, float((e / t2).max()))
    return worst


DT = ["bfloat16", "float16"]


def dtype_of(name):
    import torch
    return getattr(torch, name)


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("sizes,pre,suf,Hq,Hkv,page", [
    ([1], [1], [0], 1, 1, 1),
    ([1], [0], [1], 4, 2, 16),
    ([2, 0, 3], [5, 9, 0], [0, 1, 0, 17, 33], 8, 2, 16),
    ([12], [300], [1, 2, 3, 4] * 3, 16, 4, 16),
    ([5, 1, 9], [129, 64, 1000], [0, 70, 16] * 5, 14, 2, 20),
    ([33], [257], [3] * 33, 8, 1, 32),
    ([3, 4], [127, 383], [64] * 7, 9, 3, 128),
    ([2], [40], [5, 6], 6, 6, 8),
    ([1, 1], [700, 20], [0, 5], 40, 1, 5),
])
def test_matches_definition(dt, D, sizes, pre, suf, Hq, Hkv, page):
    torch, dev = torch_dev()
    s = make(sizes, pre, suf, Hq, Hkv, D, page, dtype_of(dt), seed=len(suf) + D)
    poison(s)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    check(s, call(s, dev_status=status))
    assert int(status.item()) == 0


@pytest.mark.parametrize("page", [16, 48, 64, 256])
def test_long_prefixes(page):
    """Work split over many workers, and shared blocks of more than 128 pairs."""
    torch, dev = torch_dev()
    s = make([40, 3, 150], [5000, 9000, 2100], [2, 9, 1] * 64 + [7], 8, 2, 128, page,
             torch.bfloat16, seed=page)
    poison(s)
    check(s, call(s), rows=list(range(0, 193, 7)) + [39, 40, 42, 43, 192])


@pytest.mark.parametrize("D,page", [(256, 64), (128, 64), (64, 20)])
@pytest.mark.parametrize("suf", [[3, 0, 9, 100], [1, 2, 0, 3]])
def test_few_rows_over_long_prefixes(D, page, suf):
    """A hundred partials for a row: several warps join them."""
    s = make([2, 1, 1], [9990, 0, 6011], suf, 14, 2, D, page, dtype_of("float16"), seed=D)
    poison(s)
    check(s, call(s))


@pytest.mark.parametrize("sizes,pre", [
    ([33], [4999]),                     # two blocks of a prefix's pairs
    ([95], [2111]), ([160], [3001]),    # three, five
    ([250], [4090]), ([310], [1000]),   # eight, ten
    ([64, 60, 5], [1500, 700, 900]),    # blocks of several prefixes, one of a single block
    ([130, 8, 8], [6000, 0, 0]),        # groups without tokens beside
])
@pytest.mark.parametrize("own", [80, 900])
def test_several_blocks_of_a_prefix(sizes, pre, own):
    """As many blocks as divide the workers or not: some may be left out, half of
    them with long own caches."""
    R = sum(sizes)
    s = make(sizes, pre, np.arange(R) * 157 % own, 32, 8, 128, 32, dtype_of("bfloat16"), seed=R)
    poison(s)
    check(s, call(s), rows=sorted(set(range(0, R, 5)) | {R - 1}))


@pytest.mark.parametrize("page", [16, 128, 20])
def test_many_short_groups(page):
    """Every worker has many items, most of them of one tile."""
    rng = np.random.default_rng(page)
    n = 700
    s = make(rng.integers(0, 4, n), rng.integers(0, 400, n), None, 8, 4, 128, page,
             dtype_of("bfloat16"), seed=page, own=False)
    poison(s)
    check(s, call(s), rows=range(0, s["q"].shape[0], 9))


def test_long_own_tokens():
    """Few rows with long own caches: their stretches are split too."""
    torch, dev = torch_dev()
    for dt, D in (("bfloat16", 128), ("float16", 64)):
        s = make([2, 1], [100, 0], [3000, 1, 4097], 8, 2, D, 16, dtype_of(dt), seed=D)
        poison(s)
        check(s, call(s))


@pytest.mark.parametrize("order", ["hnd", "pnh"])
@pytest.mark.parametrize("page", [16, 12])
def test_cache_layouts(order, page):
    s = make([7, 2], [200, 77], [3] * 9, 8, 4, 128, page, dtype_of("bfloat16"), order=order)
    poison(s)
    check(s, call(s))


def test_strides_of_queries_and_outputs():
    torch, dev = torch_dev()
    s = make([4, 5], [90, 150], [4] * 9, 8, 2, 64, 16, torch.bfloat16)
    wide = torch.zeros((9, 11, 80), dtype=torch.bfloat16, device=dev)
    wide[:, 1:9, 8:72] = s["q"]
    y = torch.full((8, 9, 72), 5.0, dtype=torch.bfloat16, device=dev).permute(1, 0, 2)
    want = call(s)["out"]
    o = call(dict(s, q=wide[:, 1:9, 8:72]),
             out={"out": y[..., :64], "lse": torch.empty((9, 8), device=dev)})
    assert torch.equal(o["out"], want) and bool((y[..., 64:] == 5.0).all())


def test_without_own_tokens_without_groups_without_lse():
    torch, dev = torch_dev()
    s = make([4, 2], [90, 0], [0] * 6, 4, 2, 128, 16, torch.float16, own=False)
    o = call(s, lse=False)
    assert "lse" not in o
    check(s, o)
    s = make([3], [0], [5, 0, 40], 4, 2, 128, 16, torch.float16)
    o = call(dict(s, pt=s["pt"][:0], pl=s["pl"][:0], off=s["off"][:1]))
    check(s, o)


@pytest.mark.parametrize("spread", [0.0, 6.0])
def test_flat_and_peaked_scores(spread):
    """Equal scores, and scores in the hundreds: one weight is nearly 1."""
    s = make([6, 30], [400, 900], [9] * 36, 8, 2, 128, 16, dtype_of("bfloat16"), spread=spread)
    check(s, call(s), rows=range(0, 36, 3))
    check(s, call(s, scale=0.5), scale=0.5, rows=range(0, 36, 5))


def test_rising_scores():
    """Every token scores higher than those before: the maximum never rests."""
    torch, dev = torch_dev()
    s = make([20], [1500], [40] * 20, 8, 2, 128, 16, torch.bfloat16)
    page = s["k"].shape[1]
    t = torch.arange(1500, device=dev)
    s["k"][s["pt"][0][t // page].long(), t % page] = \
        (t.float() * 0.02)[:, None, None].to(torch.bfloat16)
    s["q"] = s["q"].abs() * 0.3
    check(s, call(s), rows=range(0, 20, 4))


@pytest.mark.parametrize("D,Hq,Hkv,rows,suf", [
    (128, 32, 8, 700, 6), (64, 8, 8, 900, 9),   # several key/value heads to a warp
    (256, 24, 8, 500, 5),
    (128, 32, 8, 20, 6),                        # a warp each
    (128, 32, 8, 60, 200), (256, 8, 4, 9, 70),  # a kernel of their own for own tokens
])
def test_infinite_values_stay_with_their_head(D, Hq, Hkv, rows, suf):
    """An infinity or NaN among a head's values reaches the rows and heads that
    read it, and no others."""
    torch, dev = torch_dev()
    sizes = [rows // 2, rows - rows // 2]
    s = make(sizes, [70, 33], [suf] * rows, Hq, Hkv, D, 16, torch.float16, seed=rows)
    want = call(s)["out"].clone()
    M = Hq // Hkv
    hit = torch.zeros((rows, Hq), dtype=torch.bool, device=dev)
    v = s["v"]
    for r, h, x in ((0, 1, float("inf")), (rows - 1, 0, float("nan")),
                    (rows // 3, Hkv - 1, float("-inf")), (rows // 3 + 1, 2, float("nan"))):
        v[int(s["t"][r, (suf - 1) // 16]), (suf - 1) % 16, h] = x
        hit[r, h * M:(h + 1) * M] = True
    v[int(s["pt"][1, 1]), 3, 3] = float("inf")      # a token of the second prefix
    hit[sizes[0]:, 3 * M:4 * M] = True
    got = call(s)["out"]
    assert bool(torch.isfinite(got[~hit]).all())
    assert torch.equal(got[~hit], want[~hit])
    assert not bool(torch.isfinite(got[hit]).any())


@pytest.mark.parametrize("D,page,rows,suf", [(128, 16, 700, 6), (64, 20, 30, 90), (256, 16, 40, 3)])
def test_queries_that_are_no_numbers_stay_in_their_row(D, page, rows, suf):
    torch, dev = torch_dev()
    s = make([rows], [500], [suf] * rows, 16, 4, D, page, torch.bfloat16, seed=rows)
    s["q"][3, 5] = float("nan")
    s["q"][rows - 2, 0, 7] = float("inf")
    keep = torch.ones((rows, 16), dtype=torch.bool, device=dev)
    keep[3, 5] = keep[rows - 2, 0] = False
    got = call(s)["out"]
    assert bool(torch.isfinite(got[keep]).all())
    assert not bool(torch.isfinite(got[~keep]).any())
    check(s, call(s), rows=[0, 2, 4, rows // 2, rows - 3, rows - 1])


def test_rows_in_no_group():
    torch, dev = torch_dev()
    s = make([3, 4, 2], [50, 60, 70], [5] * 9, 4, 2, 64, 16, torch.bfloat16)
    inner = dict(s, off=s["off"][1:3].clone(), pl=s["pl"][1:2].clone(), pt=s["pt"][1:2].clone())
    s["pre"] = np.array([0, 60, 0])
    check(s, call(inner))


def test_bad_pages_and_lengths_are_flagged():
    torch, dev = torch_dev()
    s = make([3, 4], [50, 60], [20] * 7, 4, 2, 128, 16, torch.bfloat16)
    status = torch.zeros(1, dtype=torch.int32, device=dev)

    def flags(**kw):
        status.zero_()
        o = call(dict(s, **kw), dev_status=status)
        assert bool(torch.isfinite(o["out"].float()).all())
        return int(status.item())

    pages = s["k"].shape[0]
    for bad in (-1, pages, 2 ** 31 - 1):
        pt, t = s["pt"].clone(), s["t"].clone()
        pt[1, 2], t[4, 1] = bad, bad
        assert flags(pt=pt) == ssd.DEV_BAD_PAGE
        assert flags(t=t) == ssd.DEV_BAD_PAGE
    full = s["pt"].clamp(0, pages - 1)  # clamped lengths reach every column
    own = s["t"].clamp(0, pages - 1)
    for n in (-1, 10 ** 6):
        pl, l = s["pl"].clone(), s["l"].clone()
        pl[0], l[3] = n, n
        assert flags(pl=pl, pt=full) == ssd.DEV_BAD_LENGTH
        assert flags(l=l, t=own) == ssd.DEV_BAD_LENGTH
    for off in ([0, 5, 2], [0, 3, 8], [-1, 3, 7], [7, 0, 7]):
        assert flags(off=i32(off)) == ssd.DEV_BAD_LENGTH


def test_page_read_as_zeros():
    torch, dev = torch_dev()
    s = make([2], [40], [20, 9], 2, 1, 64, 8, torch.float16)
    s["pt"][0, 3] = -5
    got = call(s)
    # the same with a page of zeros in its place
    free = [p for p in range(s["k"].shape[0])
            if p not in s["pt"][0].tolist() and p not in s["t"].flatten().tolist()][0]
    s["k"][free] = 0
    s["v"][free] = 0
    s["pt"][0, 3] = free
    want = call(s)
    assert torch.equal(got["out"], want["out"]) and torch.equal(got["lse"], want["lse"])


def test_same_twice_streams_and_graph():
    torch, dev = torch_dev()
    s = make([30, 6], [3000, 500], [9] * 36, 8, 2, 128, 16, torch.bfloat16)
    a, b = call(s), call(s)
    assert torch.equal(a["out"], b["out"]) and torch.equal(a["lse"], b["lse"])
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    c = call(s, stream=st)
    st.synchronize()
    assert torch.equal(a["out"], c["out"])
    out = call(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(s, out=out)
    s["pl"].copy_(i32([1234, 77]))
    s["pre"] = np.array([1234, 77])
    g.replay()
    check(s, out, rows=range(0, 36, 5))


def test_refusals():
    torch, dev = torch_dev()
    s = make([2], [40], [3, 4], 4, 2, 64, 16, torch.bfloat16)
    call(s)
    for kw in (dict(q=s["q"].float()), dict(q=s["q"].half()), dict(q=s["q"].cpu()),
               dict(q=s["q"][0]), dict(k=s["k"][..., :32]), dict(v=s["v"][:1]),
               dict(k=s["k"].cpu(), v=s["v"].cpu()), dict(pl=s["pl"].long()),
               dict(off=s["off"][:1]), dict(pt=s["pt"].long()), dict(l=None), dict(t=s["t"][:1]),
               dict(q=s["q"][:, :3]), dict(q=s["q"].transpose(1, 2)), dict(l=s["l"][:1])):
        with pytest.raises(ssd.SSDError):
            call(dict(s, **kw))
    with pytest.raises(ssd.SSDError):
        call(s, scale=float("nan"))
    with pytest.raises(ssd.SSDError):
        call(s, workspace=torch.empty(256, dtype=torch.uint8, device=dev))
