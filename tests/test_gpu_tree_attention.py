"""tree_attention against the definition in float64, sequence by sequence.

Tolerance, from the formulas.  A score is a sum of D exact products, scaled,
and lessened by a maximum, in float32: with S the largest scale * sum |q k| of
the row it is off by at most rs = (D + 4) 2^-23 S + 2^-21 (the last term: the
exponential).  A weight is rounded to the type (eps / 2) and its sums run over
n tokens in float32 (n 2^-23); with A = sum p |v| over the normalised weights
  |out - exact| <= A (eps/2 + 2 rs + (n + 8) 2^-23) + eps/2 |exact|,
and for float16, whose small weights lose steps of 2^-24, half a step of each
weight more (its largest weight may be up to 2^8, so the sums are at least as
large and the steps no larger beside them).
|lse - exact| <= rs + n 2^-24 + 2^-21 + 2^-23 |exact|.
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


def parents(kind, N, seed=0):
    if kind == "chain":
        return None
    if kind == "binary":
        return [(u - 1) // 2 if u else -1 for u in range(N)]
    if kind == "star":
        return [0 if u else -1 for u in range(N)]
    rng = np.random.default_rng(seed)
    return [int(rng.integers(0, u)) if u else -1 for u in range(N)]


def sees(parent, N):
    """[u, v]: v is on the path to u."""
    ok = np.zeros((N, N), bool)
    for u in range(N):
        v = u
        while v >= 0:
            ok[u, v] = True
            v = v - 1 if parent is None else parent[v]
    return ok


def make(lens, N, Hq, Hkv, D, page, dtype, kind="chain", seed=0, order="nhd", spread=1.0, spare=3,
         slack=2):
    torch, dev = torch_dev()
    rng = np.random.default_rng(seed)
    gen = torch.Generator(device=dev).manual_seed(seed)
    lens = np.asarray(lens)
    B = len(lens)
    n = -(-lens // page)
    total = int(n.sum()) + spare
    ids = rng.permutation(total)
    # unused columns hold what is no page: they are never read
    table = np.full((B, max(1, int(n.max(initial=0))) + slack), -12345)
    table[np.arange(table.shape[1]) < n[:, None]] = ids[:n.sum()]
    shape = {"nhd": (total, page, Hkv, D), "hnd": (total, Hkv, page, D),
             "pnh": (page, total, Hkv, D)}[order]
    perm = {"nhd": (0, 1, 2, 3), "hnd": (0, 2, 1, 3), "pnh": (1, 0, 2, 3)}[order]

    def normal(*shape, by=1.0):
        return (torch.randn(shape, generator=gen, device=dev) * by).to(dtype)

    return dict(q=normal(B, N, Hq, D, by=spread), k=normal(B, N, Hkv, D, by=spread),
                v=normal(B, N, Hkv, D), kc=normal(*shape, by=spread).permute(perm),
                vc=normal(*shape).permute(perm), t=i32(table), l=i32(lens), lens=lens,
                parent=parents(kind, N, seed))


def poison(s):
    """NaN in every cache entry that no sequence reads."""
    torch, dev = torch_dev()
    pages, page = s["kc"].shape[:2]
    used = torch.zeros((pages, page), dtype=torch.bool, device=dev)
    for i, n in enumerate(s["lens"]):
        t = torch.arange(int(n), device=dev)
        used[s["t"][i][t // page].long(), t % page] = True
    for c in (s["kc"], s["vc"]):
        c[~used] = float("nan")


def call(s, **kw):
    return ssd.tree_attention(s["q"], s["k"], s["v"], s["kc"], s["vc"], s["t"], s["l"],
                              parent=s["parent"], **kw)


def check(s, o, scale=None, seqs=None):
    torch, dev = torch_dev()
    B, N, Hq, D = s["q"].shape
    page, Hkv = s["kc"].shape[1:3]
    M = Hq // Hkv
    scale = D ** -0.5 if scale is None else scale
    eps = torch.finfo(s["q"].dtype).eps
    half = s["q"].dtype == torch.float16
    assert o["out"].shape == (B, N, Hq, D) and o["out"].dtype == s["q"].dtype
    hidden = ~torch.from_numpy(sees(s["parent"], N)).to(dev)[None, None]
    for b in range(B) if seqs is None else seqs:
        n = int(s["lens"][b])
        t = torch.arange(n, device=dev)
        at = (s["t"][b][t // page].long(), t % page)
        k, v = (torch.cat([c[at], x[b]]).double() for c, x in ((s["kc"], s["k"]), (s["vc"], s["v"])))
        x = s["q"][b].double().view(N, Hkv, M, D)
        sc = torch.einsum("uhmd,thd->hmut", x, k) * scale
        big = torch.einsum("uhmd,thd->hmut", x.abs(), k.abs()) * abs(scale)
        sc[..., n:].masked_fill_(hidden, -math.inf)
        big[..., n:].masked_fill_(hidden, 0.0)
        rs = (D + 4) * 2.0 ** -23 * big.amax(-1, keepdim=True) + 2.0 ** -21
        p = torch.softmax(sc, -1)
        want = torch.einsum("hmut,thd->hmud", p, v)
        A = torch.einsum("hmut,thd->hmud", p, v.abs())
        tol = A * (eps / 2 + 2 * rs + (n + N + 8) * 2.0 ** -23) + eps / 2 * want.abs()
        if half:
            tol = tol + 2.0 ** -25 * (v.abs().sum(0)[:, None, None] + 1)
        err = (o["out"][b].double().view(N, Hkv, M, D).permute(1, 2, 0, 3) - want).abs()
        assert bool((err <= tol).all()), (b, float((err / tol).max()))
        if "lse" in o:
            ref = torch.logsumexp(sc, -1)
            e = (o["lse"][b].double().view(N, Hkv, M).permute(1, 2, 0) - ref).abs()
            t2 = rs[..., 0] + (n + N) * 2.0 ** -24 + 2.0 ** -21 + 2.0 ** -23 * ref.abs()
            assert bool((e <= t2).all()), (b, float((e / t2).max()))


def dtype_of(name):
    import torch
    return getattr(torch, name)


@pytest.mark.parametrize("dt", ["bfloat16", "float16"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("lens,N,Hq,Hkv,page,kind", [
    ([0], 1, 1, 1, 1, "chain"),
    ([1], 1, 4, 2, 16, "chain"),
    ([0, 5, 0], 3, 8, 2, 16, "binary"),
    ([300, 128, 127, 129], 5, 16, 4, 16, "chain"),
    ([129, 64, 1000], 7, 14, 2, 20, "binary"),
    ([257], 33, 8, 1, 32, "random"),
    ([127, 383], 17, 9, 3, 128, "star"),
    ([40, 63, 64, 65], 2, 6, 6, 8, "chain"),
    ([700, 20], 9, 40, 1, 5, "random"),
    ([60, 0, 500], 64, 8, 2, 16, "random"),
    ([30, 250], 130, 4, 2, 64, "random"),
    ([77], 256, 3, 1, 256, "chain"),
    ([129], 255, 4, 4, 48, "binary"),
])
def test_matches_definition(dt, D, lens, N, Hq, Hkv, page, kind):
    torch, dev = torch_dev()
    s = make(lens, N, Hq, Hkv, D, page, dtype_of(dt), kind, seed=N + D)
    poison(s)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    check(s, call(s, dev_status=status))
    assert int(status.item()) == 0


@pytest.mark.parametrize("page,D", [(16, 128), (20, 128), (64, 64), (12, 64), (32, 256), (5, 256)])
@pytest.mark.parametrize("lens,N,Hq", [
    ([9000], 4, 8), ([5000, 12000], 16, 8), ([4000, 1, 3000], 40, 8), ([6000], 100, 16)])
def test_long_caches(page, D, lens, N, Hq):
    """Work split over many workers, several blocks of pairs."""
    s = make(lens, N, Hq, 2, D, page, dtype_of("bfloat16"), "random", seed=page)
    poison(s)
    check(s, call(s))


@pytest.mark.parametrize("page", [16, 20])
@pytest.mark.parametrize("N,D", [(1, 128), (3, 64), (48, 128), (2, 256)])
def test_many_sequences(page, N, D):
    """Every worker has many items, most of them of a few tiles."""
    rng = np.random.default_rng(page)
    s = make(rng.integers(0, 500, 500), N, 8, 4, D, page, dtype_of("bfloat16"), "random",
             seed=page)
    poison(s)
    check(s, call(s), seqs=range(0, 500, 7))


@pytest.mark.parametrize("order", ["hnd", "pnh"])
@pytest.mark.parametrize("page", [16, 12])
@pytest.mark.parametrize("D", [128, 256])
def test_cache_layouts(order, page, D):
    s = make([200, 77, 0], 7, 8, 4, D, page, dtype_of("bfloat16"), "binary", order=order)
    poison(s)
    check(s, call(s))


@pytest.mark.parametrize("Hq,Hkv,N,lens", [(160, 1, 3, [700, 0]), (144, 1, 1, [5000]), (48, 3, 30, [90]),
                                          (64, 1, 256, [300]), (7, 7, 200, [1000, 2]),
                                          (33, 11, 5, [64] * 9)])
@pytest.mark.parametrize("D,page", [(64, 16), (128, 48), (256, 32)])
def test_head_counts(Hq, Hkv, N, lens, D, page):
    """Groups of heads of any size, more blocks of pairs than stand side by side."""
    s = make(lens, N, Hq, Hkv, D, page, dtype_of("bfloat16"), "random", seed=Hq)
    poison(s)
    check(s, call(s))


@pytest.mark.parametrize("Hq,Hkv,N,lens", [(56, 8, 57, [3, 900, 0]), (15, 3, 52, [4000]), (9, 3, 100, [70, 1]),
                                          (24, 2, 23, [260, 5, 0]), (40, 2, 13, [33] * 5), (96, 2, 9, [500]),
                                          (200, 2, 4, [100, 2000]), (127, 1, 2, [64])])
@pytest.mark.parametrize("D,page", [(64, 16), (128, 16), (128, 20), (256, 64)])
@pytest.mark.parametrize("scale", [None, -0.11, 0.0])
def test_groups_that_do_not_divide_a_block(Hq, Hkv, N, lens, D, page, scale):
    """Blocks of whole nodes with rows left empty, or nodes shared by two blocks; queries by boxes and row
    by row; the output in the queries' place."""
    s = make(lens, N, Hq, Hkv, D, page, dtype_of("bfloat16"), "random", seed=N)
    poison(s)
    kw = {} if scale is None else {"scale": scale}
    o = call(s, **kw)
    check(s, o, **kw)
    q = s["q"].clone()
    again = call(dict(s, q=q), out={"out": q}, **kw)
    assert (again["out"] == o["out"]).all() and (again["lse"] == o["lse"]).all()


@pytest.mark.parametrize("N", [1, 31, 32, 33, 64, 65, 97, 129])
@pytest.mark.parametrize("D,page", [(64, 16), (128, 16), (128, 20), (256, 64)])
def test_lengths_about_multiples_of_32(N, D, page):
    """Tiles of which some of the 32s hold no token; the slots' other rows are those of earlier tiles."""
    lens = [0, 1, 31, 32, 33, 63, 64, 65, 95, 96, 97, 127, 128, 129, 160, 161, 224, 255, 257, 300] * 4
    s = make(lens, N, 4, 4, D, page, dtype_of("float16"), "random", seed=D)
    poison(s)
    check(s, call(s))


def test_keys_and_values_with_a_layout_each_and_tables_in_wider_rows():
    torch, dev = torch_dev()
    s = make([200, 77, 500], 7, 8, 4, 128, 16, torch.bfloat16, "binary")
    poison(s)
    want = {k: v.clone() for k, v in call(s).items()}
    wide = torch.full((3, 60), 3, dtype=torch.int32, device=dev)
    wide[:, 9:9 + s["t"].shape[1]] = s["t"]
    vc = s["vc"].permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3)
    k = s["k"].permute(2, 0, 1, 3).contiguous().permute(1, 2, 0, 3)
    got = call(dict(s, vc=vc, k=k, t=wide[:, 9:9 + s["t"].shape[1]]))
    assert torch.equal(got["out"], want["out"]) and torch.equal(got["lse"], want["lse"])


@pytest.mark.parametrize("page", [4, 6, 24, 40, 192, 384])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_pages_of_any_size(page, D):
    s = make([1000, 7, 385], 6, 8, 2, D, page, dtype_of("float16"), "random", seed=page)
    poison(s)
    check(s, call(s))


@pytest.mark.parametrize("N", [1, 5])
def test_pieces_of_one_projection_and_strided_outputs(N):
    torch, dev = torch_dev()
    s = make([90, 150, 3], N, 8, 2, 64, 16, torch.bfloat16, "binary")
    want = {k: v.clone() for k, v in call(s).items()}
    qkv = torch.zeros((3, N, 12, 72), dtype=torch.bfloat16, device=dev)
    pieces = dict(q=qkv[:, :, :8, :64], k=qkv[:, :, 8:10, :64], v=qkv[:, :, 10:, :64])
    for n, x in pieces.items():
        x.copy_(s[n])
    y = torch.full((N, 8, 3, 72), 5.0, dtype=torch.bfloat16, device=dev).permute(2, 0, 1, 3)
    o = call(dict(s, **pieces), out={"out": y[..., :64]})
    assert torch.equal(o["out"], want["out"]) and torch.equal(o["lse"], want["lse"])
    assert bool((y[..., 64:] == 5.0).all())
    one = s["q"][:1].expand(3, N, 8, 64)  # a stride of zero
    got = call(dict(s, q=one, k=s["k"][:1].expand_as(s["k"])))
    check(dict(s, q=one.contiguous(), k=s["k"][:1].repeat(3, 1, 1, 1)), got)


@pytest.mark.parametrize("N,lens", [(4, [90, 500]), (40, [3000, 20])])
def test_in_place(N, lens):
    torch, dev = torch_dev()
    s = make(lens, N, 8, 2, 128, 16, torch.bfloat16, "random")
    want = call(s)["out"].clone()
    q = s["q"].clone()
    assert torch.equal(call(dict(s, q=q), out={"out": q})["out"], want)


def test_without_lse_without_columns():
    torch, dev = torch_dev()
    s = make([0, 0], 6, 4, 2, 128, 16, torch.float16, "random")
    o = call(s)
    check(s, call(dict(s, t=s["t"][:, :0])))
    p = call(s, lse=False, out=dict(o))
    assert "lse" not in p
    check(s, p)


@pytest.mark.parametrize("spread", [0.0, 6.0])
@pytest.mark.parametrize("D", [128, 256])
def test_flat_and_peaked_scores(spread, D):
    """Equal scores, and scores in the hundreds: one weight is nearly 1."""
    s = make([400, 900], 19, 8, 2, D, 16, dtype_of("bfloat16"), "random", spread=spread)
    check(s, call(s))
    for scale in (0.5, -0.125, 0.0):
        check(s, call(s, scale=scale), scale=scale)


@pytest.mark.parametrize("D,N", [(128, 5), (128, 60), (256, 5)])
def test_rising_scores(D, N):
    """Every token scores higher than those before: the maximum never rests."""
    torch, dev = torch_dev()
    s = make([1500], N, 8, 2, D, 16, torch.bfloat16)
    t = torch.arange(1500, device=dev)
    s["kc"][s["t"][0][t // 16].long(), t % 16] = (t.float() * 0.02)[:, None, None].to(torch.bfloat16)
    s["q"] = s["q"].abs() * 0.3
    check(s, call(s))


BAD = [float("nan"), float("inf"), float("-inf")]


@pytest.mark.parametrize("page", [16, 20])
@pytest.mark.parametrize("N,lens,Hq,D", [(11, [40, 300], 8, 128), (70, [3000, 10], 8, 128),
                                         (11, [2000, 30], 8, 256), (9, [100, 50], 4, 64),
                                         (200, [30, 700], 4, 64)])
def test_values_off_the_path_have_no_effect(page, N, lens, Hq, D):
    """Infinities and NaN among a node's keys and values reach the nodes below it alone."""
    torch, dev = torch_dev()
    s = make(lens, N, Hq, 2, D, page, torch.bfloat16, "binary", seed=N)
    want = {k: v.clone() for k, v in call(s).items()}
    ok = torch.from_numpy(sees(s["parent"], N)).to(dev)
    M = Hq // 2
    for i, x in enumerate(BAD):
        for name in ("k", "v"):
            z = s[name].clone()
            node = N // 2 + i
            z[1, node, 1, 3] = x
            z[0, N - 1, 0] = x          # a leaf
            got = call(dict(s, **{name: z}))
            hit = torch.zeros((2, N, Hq), dtype=torch.bool, device=dev)
            hit[1, ok[:, node], M:] = True
            hit[0, N - 1, :M] = True
            for key in ("out", "lse"):
                assert torch.equal(got[key][~hit], want[key][~hit]), (x, name, key)
            if name == "v":             # every weight on a path is positive
                part = got["out"][hit].float()
                assert bool((~torch.isfinite(part)).any(-1).all())
                if math.isinf(x):
                    assert bool((part[~torch.isfinite(part)] == x).all())
                dim = torch.arange(D, device=dev) != 3
                assert torch.equal(got["out"][1, ok[:, node], M:][..., dim],
                                   want["out"][1, ok[:, node], M:][..., dim])
            elif math.isnan(x):
                assert bool(torch.isnan(got["out"][hit].float()).all())


def test_queries_that_are_no_numbers_stay_in_their_row():
    torch, dev = torch_dev()
    s = make([500, 40], 9, 16, 4, 128, 16, torch.bfloat16, "random")
    want = call(s)["out"].clone()
    s["q"][0, 3, 5] = float("nan")
    s["q"][1, 7, 0, 7] = float("inf")
    keep = torch.ones((2, 9, 16), dtype=torch.bool, device=dev)
    keep[0, 3, 5] = keep[1, 7, 0] = False
    got = call(s)["out"]
    assert torch.equal(got[keep], want[keep])
    assert not bool(torch.isfinite(got[~keep]).any())


@pytest.mark.parametrize("N", [3, 200])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_no_scores_and_values_that_are_no_numbers(N, D):
    """Every score of a row is -inf, and a value on its path is no number: zeros."""
    torch, dev = torch_dev()
    s = make([0, 0], N, 4, 2, D, 16, torch.bfloat16, "chain")
    s["q"].fill_(1.0)
    s["k"][0].fill_(-math.inf)
    s["v"][0, 1, 0, ::3] = math.inf
    s["v"][0, 2, 1, 5] = math.nan
    o = call(s)
    assert bool((o["out"][0] == 0).all()) and bool((o["lse"][0] == -math.inf).all())
    check(s, o, seqs=[1])


def test_infinite_keys_of_every_token():
    """Scores of -inf alone: zeros, and -inf."""
    torch, dev = torch_dev()
    s = make([0], 1, 2, 1, 64, 16, torch.float16)
    s["q"][:] = 1.0
    s["k"][:] = float("-inf")
    o = call(s)
    assert bool((o["out"] == 0).all()) and bool((o["lse"] == -math.inf).all())


@pytest.mark.parametrize("page", [16, 20])
def test_bad_pages_and_lengths_are_flagged(page):
    torch, dev = torch_dev()
    s = make([50, 60], 4, 4, 2, 128, page, torch.bfloat16)
    status = torch.zeros(1, dtype=torch.int32, device=dev)

    def flags(**kw):
        status.zero_()
        o = call(dict(s, **kw), dev_status=status)
        assert bool(torch.isfinite(o["out"].float()).all())
        return int(status.item())

    pages = s["kc"].shape[0]
    for bad in (-1, pages, 2 ** 31 - 1, -2 ** 31):
        t = s["t"].clone()
        t[1, 2] = bad
        assert flags(t=t) == ssd.DEV_BAD_PAGE
        # the same with a page of zeros in its place
        got = {k: v.clone() for k, v in call(dict(s, t=t)).items()}
        free = [p for p in range(pages) if p not in s["t"].flatten().tolist()][0]
        s["kc"][free] = 0
        s["vc"][free] = 0
        t[1, 2] = free
        want = call(dict(s, t=t))
        assert torch.equal(got["out"], want["out"]) and torch.equal(got["lse"], want["lse"])
    full = s["t"].clamp(0, pages - 1)  # clamped lengths reach every column
    for n in (-1, 10 ** 6, -2 ** 31, 2 ** 31 - 1):
        l = s["l"].clone()
        l[0] = n
        assert flags(l=l, t=full) == ssd.DEV_BAD_LENGTH
        lens = np.array([0 if n < 0 else full.shape[1] * page, 60])
        check(dict(s, t=full, lens=lens), call(dict(s, l=l, t=full)))


def test_same_twice_streams_and_graphs():
    torch, dev = torch_dev()
    s = make([3000, 500, 40], 12, 8, 2, 128, 16, torch.bfloat16, "random")
    a, b = call(s), call(s)
    assert torch.equal(a["out"], b["out"]) and torch.equal(a["lse"], b["lse"])
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    c = call(s, stream=st)
    d = call(s)                                 # beside it
    st.synchronize()
    assert torch.equal(a["out"], c["out"]) and torch.equal(a["out"], d["out"])
    out = call(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(s, out=out)
    s["l"].copy_(i32([1234, 77, 0]))
    s["lens"] = np.array([1234, 77, 0])
    for _ in range(2):
        out["out"].zero_()
        g.replay()
        check(s, out)


@pytest.mark.parametrize("N,Hq,D,lens", [(5, 8, 128, [900] * 60), (40, 8, 128, [700, 1500] * 20),
                                         (7, 8, 256, [500] * 40), (9, 4, 64, [1100] * 50)])
def test_same_bits_beside_other_work(N, Hq, D, lens):
    """Items of two stretches, whose workers begin and end at any time."""
    torch, dev = torch_dev()
    s = make(lens, N, Hq, 2, D, 16, torch.bfloat16, "random", seed=N)
    first = {k: v.clone() for k, v in call(s).items()}
    check(s, first, seqs=range(0, len(lens), 9))
    out, busy = {}, torch.randn((4096, 4096), device=dev)
    side = torch.cuda.Stream()
    for i in range(60):
        if i % 3 == 0:      # work beside it, so that its CTAs begin at other times
            with torch.cuda.stream(side):
                busy = (busy @ busy).clamp(-1, 1)
        out.get("out", first["out"][:0]).zero_()
        call(s, out=out)
        assert torch.equal(out["out"], first["out"]) and torch.equal(out["lse"], first["lse"]), i
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(s, out=out)
    for i in range(30):
        out["out"].zero_()
        g.replay()
        assert torch.equal(out["out"], first["out"]) and torch.equal(out["lse"], first["lse"]), i


def test_graphs_with_one_workspace_take_turns():
    torch, dev = torch_dev()
    ws = torch.empty(1 << 26, dtype=torch.uint8, device=dev)
    cases = [make([3000, 500], 12, 8, 2, 128, 16, torch.bfloat16, "random"),
             make([70] * 40, 3, 8, 4, 64, 20, torch.float16)]
    outs, graphs = [{}, {}], []
    for s, o in zip(cases, outs):
        call(s, workspace=ws, out=o)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(s, workspace=ws, out=o)
        graphs.append(g)
    for _ in range(3):
        for s, o, g in zip(cases, outs, graphs):
            o["out"].zero_()
            g.replay()
            check(s, o)


def test_threads_at_once():
    """Calls of several threads, each on a stream of its own."""
    import threading

    torch, dev = torch_dev()
    cases = [make([900, 20 * i], 3 + i, 8, 2, (64, 128, 256)[i % 3], 16, torch.bfloat16, "random",
                  seed=i) for i in range(6)]
    want = [call(s) for s in cases]
    torch.cuda.synchronize()
    got, errors = [None] * 6, []

    def work(i):
        try:
            st = torch.cuda.Stream()
            for _ in range(20):
                got[i] = call(cases[i], stream=st)
            st.synchronize()
        except Exception as e:   # shown by the main thread
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(6)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors
    for g, w in zip(got, want):
        assert torch.equal(g["out"], w["out"]) and torch.equal(g["lse"], w["lse"])


def test_offsets_beyond_32_bits():
    """A cache of more than 2^32 elements: pages at its end."""
    torch, dev = torch_dev()
    s = make([100, 33], 4, 8, 2, 128, 16, torch.bfloat16, "random")
    want = {k: v.clone() for k, v in call(s).items()}
    pages = s["kc"].shape[0]
    last = (1 << 32) // (16 * 2 * 128) + 7
    for page in (16, None):
        big = {}
        for name in ("kc", "vc"):
            big[name] = torch.zeros((last + pages, 16, 2, 128), dtype=torch.bfloat16, device=dev)
            big[name][last:] = s[name]
        if page is None:                # strides that no box takes
            big["k"] = s["k"][:1].expand_as(s["k"])
            want = {k: v.clone() for k, v in call(dict(s, k=big["k"])).items()}
        t = torch.where(s["t"] >= 0, s["t"] + last, s["t"])
        got = call(dict(s, t=t, **big))
        assert torch.equal(got["out"], want["out"]) and torch.equal(got["lse"], want["lse"])
        del big


def test_dict_of_an_earlier_call():
    """A workspace that is too small is replaced."""
    torch, dev = torch_dev()
    out = {}
    for lens, N, D in (([30], 2, 64), ([4000, 700], 2, 64), ([30], 2, 64)):
        s = make(lens, N, 4, 2, D, 16, torch.bfloat16)
        o = {"workspace": out["workspace"]} if "workspace" in out else {}
        check(s, call(s, out=o))
        out = o


def test_refusals():
    torch, dev = torch_dev()
    s = make([40, 3], 3, 4, 2, 64, 16, torch.bfloat16, "binary")
    call(s)
    for kw in (dict(q=s["q"].float()), dict(q=s["q"].half()), dict(q=s["q"].cpu()),
               dict(q=s["q"][0]), dict(k=s["k"][..., :32]), dict(v=s["v"][:1]),
               dict(kc=s["kc"].cpu(), vc=s["vc"].cpu()), dict(l=s["l"].long()),
               dict(l=s["l"][:1]), dict(t=s["t"].long()), dict(t=s["t"][:1]),
               dict(q=s["q"][:, :, :3]), dict(q=s["q"].transpose(2, 3)),
               dict(k=s["k"].half(), v=s["v"].half()), dict(parent=[-1, 0]),
               dict(parent=[-1, 1, 0]), dict(parent=[-1, 0, 2]), dict(parent=[0, 0, 0]),
               dict(kc=s["kc"][:, :, :1], vc=s["vc"][:, :, :1])):
        with pytest.raises(ssd.SSDError):
            call(dict(s, **kw))
    with pytest.raises(ssd.SSDError):
        call(s, scale=float("nan"))
    with pytest.raises(ssd.SSDError):
        call(s, workspace=torch.empty(16, dtype=torch.uint8, device=dev))
    big = make([40], 257, 2, 2, 64, 16, torch.bfloat16)
    with pytest.raises(ssd.SSDError):
        call(big)


@pytest.mark.parametrize("scale", [1e39, -1e300, float("inf")])
def test_scales_beyond_float32_are_refused(scale):
    s = make([40, 3], 3, 4, 2, 64, 16, dtype_of("bfloat16"), "binary")
    with pytest.raises(ssd.SSDError):
        call(s, scale=scale)


@pytest.mark.parametrize("below", [20.3, 24.45, 25.1, 27.0])
@pytest.mark.parametrize("D,N,Hq", [(64, 1, 1), (128, 5, 4), (64, 40, 4), (128, 40, 4), (256, 3, 2)])
def test_many_small_weights_beside_a_large_one(below, D, N, Hq):
    """Two tokens with the largest score and values of 0, and 131072 whose weights are 2^-below of
    theirs and whose values are 1: what these add up to is the output.  Each worker goes through
    whole sequences, so that the largest score is kept beside the others.

    Tolerance: as above, where a half's step is at least 2^-24 beside a largest weight of at least
    2^7: with W = sum |v| (n + N at most), 2^-25 W / 2^7.
    """
    torch, dev = torch_dev()
    n, page, B = 131072, 64, 320
    kc = torch.zeros((n // page, page, 1, D), dtype=torch.float16, device=dev)
    vc = torch.ones_like(kc)
    for t in (0, 128):                   # of both streams of tiles
        kc[t // page, t % page, 0, 0], vc[t // page, t % page] = 1.0, 0.0
    q = torch.zeros((B, N, Hq, D), dtype=torch.float16, device=dev)
    q[..., 0] = 1.0
    k = torch.zeros((B, N, 1, D), dtype=torch.float16, device=dev)
    tables = torch.arange(n // page, dtype=torch.int32, device=dev).expand(B, -1).contiguous()
    scale = float(np.float32(below * math.log(2)))
    o = ssd.tree_attention(q, k, torch.ones_like(k), kc, vc, tables, i32([n] * B), scale=scale)
    w = math.exp(-scale)
    for u in {0, N - 1}:
        small = (n - 2 + u + 1) * w
        want, A = small / (2 + small), small / (2 + small)
        rs = (D + 4) * 2.0 ** -23 * scale + 2.0 ** -21
        eps = torch.finfo(torch.float16).eps
        tol = A * (eps / 2 + 2 * rs + (n + N + 8) * 2.0 ** -23) + eps / 2 * want + 2.0 ** -32 * (n + N)
        got = o["out"][:, u].double()
        assert float((got - want).abs().max()) <= tol, (float(got.min()), float(got.max()), want, tol)
        lse = scale + math.log(2 + small)
        assert float((o["lse"][:, u].double() - lse).abs().max()) <= \
            rs + (n + N) * 2.0 ** -24 + 2.0 ** -21 + 2.0 ** -23 * lse


@pytest.mark.parametrize("dt,top", [("float16", 20.4), ("float16", 24.3), ("float16", 26.7),
                                    ("float16", 27.95), ("bfloat16", 24.3), ("bfloat16", 30.95)])
@pytest.mark.parametrize("D,N,Hq", [(64, 2, 4), (128, 2, 4), (128, 70, 4), (256, 2, 4)])
@pytest.mark.parametrize("cached", [0, 700])
def test_large_scores(dt, top, D, N, Hq, cached):
    """Scores of 2^top (base 2), which float32 rounds to multiples of up to 128, equal ones alike: nodes
    with one key share their row equally, beside cached tokens that come nowhere near.

    Each row has one weight w, which the type rounds by eps / 2 and their sum does not; the sum of
    the values is off by N 2^-23 in float32, the reciprocal and its product by 2^-23 each, and the
    output is rounded by eps / 2, or a half's 2^-25:
      |out - mean| <= (eps / 2) |mean| + (eps / 2 + (N + 4) 2^-23) mean |v| + 2^-25.
    A row's weight is 2^-16 to 1 (bf16: 2^-64 to 2^64), beyond what either type rounds otherwise
    (half: normal from 2^-14, and 2^7 more here)."""
    torch, dev = torch_dev()
    t = dtype_of(dt)
    B, eps = 100, torch.finfo(t).eps
    s = make([cached] * B, N, Hq, 2, D, 16, t, seed=D)
    s["q"].fill_(200.0)
    s["k"].fill_(300.0)
    s["kc"].fill_(150.0)
    scale = 2.0 ** top / math.log2(math.e) / (200.0 * 300.0 * D)
    for sign in (1, -1):
        o = call(dict(s, q=s["q"] * sign), scale=sign * scale)
        v = s["v"].double()[:, :, torch.arange(Hq, device=dev) // (Hq // 2)]
        n = torch.arange(1, N + 1, device=dev)[:, None, None]
        mean, A = v.cumsum(1) / n, v.abs().cumsum(1) / n
        tol = eps / 2 * mean.abs() + (eps / 2 + (N + 4) * 2.0 ** -23) * A + 2.0 ** -25
        assert bool(((o["out"].double() - mean).abs() <= tol).all())
        lse = 2.0 ** top / math.log2(math.e)
        assert bool(((o["lse"] - lse).abs() <= (D + 8) * 2.0 ** -23 * lse + math.log(N)).all())


def test_large_scores_of_a_row_leave_the_others_bits():
    torch, dev = torch_dev()
    for t, N in ((torch.float16, 9), (torch.bfloat16, 40)):
        s = make([500, 40], N, 16, 4, 128, 16, t, "random")
        want = {k: call(s)[k].clone() for k in ("out", "lse")}
        s["q"][0, 3, 5] = 3e4
        keep = torch.ones((2, N, 16), dtype=torch.bool, device=dev)
        keep[0, 3, 5] = False
        got = call(s)
        for k in want:
            assert torch.equal(got[k][keep], want[k][keep])
