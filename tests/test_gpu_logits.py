"""process_logits against its definition in float64.

Tolerance, from the formula: a quotient or product, the product f*c, two
differences and a sum, each off by at most 2^-24 of a value no larger than
M = |z| max(r, 1/r) + f c + |p| + |bias|, then one rounding to the row type
(half a step, eps / 2 of the value).  Six instead of five cover the second
order terms.  Masked tokens, counts and untouched tokens are exact.
"""

import numpy as np
import pytest

import sampling_ssd_verify_gb300 as ssd
from tests.parity import i32, torch_dev

pytestmark = pytest.mark.gpu

TREE = [-1, 0, 0, 1, 1, 1, 2, 4, 4, 7, 8]


@pytest.fixture(scope="module", autouse=True)
def built():
    ssd.build()
    ssd.lib()


def expected(z, hist, hlen, plen, drafts, parent, rep, pres, freq, ids, bias, mask, fill):
    """z [B, N, V] float64; returns (out, bound, allowed) in float64."""
    B, N, V = z.shape
    out, bound = z.copy(), np.abs(z)
    allowed = np.full((B, N), V)
    for b in range(B):
        n = 0 if hist is None else min(max(int(hlen[b]), 0), hist.shape[1])
        h = np.zeros(0, int) if hist is None else hist[b, :n]
        m = 0 if plen is None else plen[b]
        for u in range(N):
            path, w = [], u
            while w > 0:
                path.append(w)
                w = parent[w]
            extra = [] if drafts is None else [drafts[b, w - 1] for w in path]
            c = np.zeros(V)
            seen = np.zeros(V, bool)
            for i, t in enumerate(h):
                if 0 <= t < V:
                    seen[t] = True
                    c[t] += i >= m
            for t in extra:
                if 0 <= t < V:
                    seen[t] = True
                    c[t] += 1
            r = 1.0 if rep is None or not (0 < rep[b] < np.inf) else float(rep[b])
            f = 0.0 if freq is None or not np.isfinite(freq[b]) else float(freq[b])
            p = 0.0 if pres is None or not np.isfinite(pres[b]) else float(pres[b])
            x = z[b, u]
            with np.errstate(invalid="ignore"):
                x = np.where(seen, np.where(x > 0, x / r, x * r), x)
            x = x - f * c - p * (c > 0)
            M = np.abs(z[b, u]) * max(r, 1 / r) + abs(f) * c + abs(p)
            if ids is not None:
                last = {int(t): float(v) for t, v in zip(ids[b], bias[b]) if 0 <= t < V}
                for t, v in last.items():
                    x[t] += v
                    M[t] += abs(v)
            if mask is not None:
                ok = mask[b % mask.shape[0], u % mask.shape[1]]
                x = np.where(ok, x, fill)
                M = np.where(ok, M, 0)
                allowed[b, u] = ok.sum()
            out[b, u], bound[b, u] = x, M
    return out, bound, allowed


def pack(mask):
    """bool [B, N, V] -> int32 words."""
    B, N, V = mask.shape
    W = (V + 31) // 32
    bits = np.zeros((B, N, W * 32), np.uint8)
    bits[..., :V] = mask
    return np.packbits(bits, axis=-1, bitorder="little").view(np.int32).reshape(B, N, W)


def check(got, want, bound, dtype):
    import torch
    eps = torch.finfo(dtype).eps
    got = got.double().cpu().numpy()
    same = (got == want) | (np.isnan(got) & np.isnan(want))
    with np.errstate(invalid="ignore"):
        err = np.abs(got - want)
    tol = (6 * 2.0 ** -24) * bound + (0 if dtype == torch.float32 else eps / 2) * np.abs(want)
    bad = ~(same | (err <= tol))
    assert not bad.any(), (np.argwhere(bad)[:5], got[bad][:5], want[bad][:5])


def make(B, N, V, H, dtype, seed, tree=False, nb=7, mask_rows=None, pad=0, shift=0):
    torch, dev = torch_dev()
    rng = np.random.default_rng(seed)
    flat = torch.from_numpy((rng.standard_normal(shift + B * N * (V + pad)) * 3).astype(np.float32))
    z = flat.to(dev).to(dtype)[shift:].view(B, N, V + pad)[..., :V]
    hot = max(1, min(V, 40))
    hist = rng.integers(0, hot, (B, H)) * 31 % V
    hlen = rng.integers(0, H + 1, B)
    plen = rng.integers(0, H + 1, B)
    drafts = rng.integers(0, hot, (B, max(N - 1, 1))) * 31 % V
    d = dict(hist=hist, hlen=hlen, plen=plen, drafts=drafts,
             rep=rng.uniform(0.7, 1.5, B).astype(np.float32),
             pres=rng.uniform(-1, 1, B).astype(np.float32),
             freq=rng.uniform(-.5, .5, B).astype(np.float32),
             ids=rng.integers(-2, V, (B, nb)) if nb else None,
             bias=rng.uniform(-5, 5, (B, nb)).astype(np.float32) if nb else None, mask=None)
    if mask_rows is not None:
        d["mask"] = rng.random((mask_rows[0], mask_rows[1], V)) < 0.3
        d["mask"][0, 0] = False       # a row that allows nothing
        d["mask"][-1, -1] = True
    return z, d, (TREE[:N] if tree else list(range(-1, N - 1)))


def call(z, d, parent, fill, **kw):
    torch, dev = torch_dev()
    f = lambda a: None if a is None else torch.from_numpy(a).to(dev)  # noqa: E731
    return ssd.process_logits(
        z, i32(d["hist"]), i32(d["hlen"]), i32(d["plen"]),
        draft_tokens=i32(d["drafts"]) if z.shape[1] > 1 else None, parent=parent,
        repetition=f(d["rep"]), presence=f(d["pres"]), frequency=f(d["freq"]),
        bias_ids=None if d["ids"] is None else i32(d["ids"]), bias=f(d["bias"]),
        mask=None if d["mask"] is None else torch.from_numpy(pack(d["mask"])).to(dev),
        fill=fill, allowed=True, **kw)


def run_case(z, d, parent, fill=ssd.MASKED_LOGIT, **kw):
    want, bound, allowed = expected(z.double().cpu().numpy(), d["hist"], d["hlen"], d["plen"],
                                    d["drafts"] if z.shape[1] > 1 else None, parent, d["rep"],
                                    d["pres"], d["freq"], d["ids"], d["bias"], d["mask"], fill)
    o = call(z, d, parent, fill, **kw)
    check(o["logits"], want, bound, z.dtype)
    np.testing.assert_array_equal(o["allowed"].cpu().numpy(), allowed)
    return o


@pytest.mark.parametrize("dt", ["bfloat16", "float32"])
@pytest.mark.parametrize("B,N,V,H,tree,mask", [
    (1, 1, 1, 1, False, None), (1, 1, 31, 3, False, (1, 1)), (2, 3, 33, 5, False, (2, 3)),
    (3, 5, 1000, 100, False, (3, 5)), (2, 11, 4099, 300, True, (2, 11)),
    (5, 11, 8192, 64, True, (1, 11)), (2, 4, 8193, 50, False, (2, 1)),
    (70, 9, 16411, 33, False, (1, 1)), (64, 11, 20000, 20, True, None),
    (3, 7, 128256, 2000, True, (3, 7)),
])
def test_matches_definition(dt, B, N, V, H, tree, mask):
    torch, dev = torch_dev()
    z, d, parent = make(B, N, V, H, getattr(torch, dt), seed=V + N, tree=tree, mask_rows=mask)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    run_case(z, d, parent, dev_status=status)
    assert int(status.item()) == 0


@pytest.mark.parametrize("dt", ["bfloat16", "float32"])
@pytest.mark.parametrize("pad,shift,out_pad", [(0, 1, 0), (3, 0, 3), (5, 2, 1), (8, 8, 0)])
def test_strides_and_alignment(dt, pad, shift, out_pad):
    """Rows at any element offset; out with another row stride than in."""
    torch, dev = torch_dev()
    B, N, V = 3, 4, 9001
    z, d, parent = make(B, N, V, 40, getattr(torch, dt), seed=5, mask_rows=(3, 4), pad=pad,
                        shift=shift)
    wide = torch.full((B, N, V + out_pad), 7.0, dtype=z.dtype, device=dev)
    run_case(z, d, parent, out={"logits": wide[..., :V]})
    assert bool((wide[..., V:] == 7.0).all())


@pytest.mark.parametrize("dt", ["bfloat16", "float32"])
def test_in_place(dt):
    torch, dev = torch_dev()
    z, d, parent = make(4, 6, 12345, 77, getattr(torch, dt), seed=9, mask_rows=(4, 6))
    new = call(z, d, parent, -1e9)["logits"].clone()
    o = call(z, d, parent, -1e9, out={"logits": z})
    assert o["logits"].data_ptr() == z.data_ptr() and torch.equal(z, new)


@pytest.mark.parametrize("dt", ["bfloat16", "float32"])
def test_infinities_nan_and_fill_values(dt):
    """Masked tokens get the fill whatever their logits; NaN and infinities of
    the others pass through."""
    torch, dev = torch_dev()
    z, d, parent = make(2, 3, 700, 30, getattr(torch, dt), seed=3, mask_rows=(2, 3))
    z = z.contiguous()
    z[:, :, ::5] = float("nan")
    z[:, :, 1::7] = float("inf")
    z[:, :, 2::11] = float("-inf")
    for fill in (float("-inf"), float(torch.finfo(z.dtype).min), 0.0):
        run_case(z, d, parent, fill=fill)


def test_no_rules_is_a_copy_and_each_rule_alone():
    torch, dev = torch_dev()
    z, d, parent = make(3, 4, 5001, 60, torch.bfloat16, seed=1, mask_rows=(3, 4))
    assert torch.equal(ssd.process_logits(z)["logits"], z)
    f = lambda a: torch.from_numpy(a).to(dev)  # noqa: E731
    z64 = z.double().cpu().numpy()
    none = dict(hist=None, hlen=None, plen=None, drafts=None, rep=None, pres=None, freq=None,
                ids=None, bias=None, mask=None)
    h = dict(hist=d["hist"], hlen=d["hlen"])
    for part, args in [
            (dict(h, rep=d["rep"]), dict(history=i32(d["hist"]), history_len=i32(d["hlen"]),
                                         repetition=f(d["rep"]))),
            (dict(h, freq=d["freq"]), dict(history=i32(d["hist"]), history_len=i32(d["hlen"]),
                                           frequency=f(d["freq"]))),
            (dict(drafts=d["drafts"], pres=d["pres"]), dict(draft_tokens=i32(d["drafts"]),
                                                            presence=f(d["pres"]))),
            (dict(ids=d["ids"], bias=d["bias"]), dict(bias_ids=i32(d["ids"]), bias=f(d["bias"]))),
            (dict(mask=d["mask"]), dict(mask=torch.from_numpy(pack(d["mask"])).to(dev)))]:
        want, bound, _ = expected(z64, **dict(none, **part), parent=parent, fill=-2.0)
        check(ssd.process_logits(z, fill=-2.0, **args)["logits"], want, bound, z.dtype)


def test_a_token_listed_twice_takes_its_last_bias():
    torch, dev = torch_dev()
    z = torch.zeros((1, 1, 100), device=dev)
    ids = i32([[5, 9, 5, -1, 9, 5]])
    bias = torch.tensor([[1., 2., 3., 4., 5., 6.]], device=dev)
    got = ssd.process_logits(z, bias_ids=ids, bias=bias)["logits"][0, 0]
    assert got[5].item() == 6 and got[9].item() == 5 and got.sum().item() == 11


def test_bad_values_are_flagged_and_left_out():
    torch, dev = torch_dev()
    z, d, parent = make(6, 3, 900, 20, torch.float32, seed=2)
    d["hist"][0, 3], d["hist"][1, 0] = -7, 900
    d["hlen"][:] = 20
    d["hlen"][2] = 21
    d["hlen"][3] = -1
    d["drafts"][4, 0] = 1 << 30
    d["rep"][0], d["rep"][1], d["rep"][2] = 0.0, np.nan, np.inf
    d["freq"][3], d["pres"][4] = np.nan, -np.inf
    d["ids"][5, 0] = 900
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    run_case(z, d, parent, dev_status=status)
    assert int(status.item()) == ssd.DEV_BAD_TOKEN | ssd.DEV_BAD_PENALTY | ssd.DEV_BAD_LENGTH


def test_tree_and_chain_agree_and_columns_for_the_root():
    torch, dev = torch_dev()
    z, d, _ = make(3, 6, 3000, 15, torch.bfloat16, seed=4)
    a = call(z, d, None, -1.0)["logits"]
    b = call(z, d, [-1, 0, 1, 2, 3, 4], -1.0)["logits"]
    d6 = dict(d, drafts=np.concatenate([np.full((3, 1), 17), d["drafts"]], 1))
    c = call(z, d6, None, -1.0)["logits"]
    assert torch.equal(a, b) and torch.equal(a, c)


def test_wide_tree():
    """256 nodes: long paths, and neighbours in index that lie far apart."""
    torch, dev = torch_dev()
    z, d, _ = make(2, 256, 211, 9, torch.float32, seed=8, mask_rows=(1, 1))
    rng = np.random.default_rng(0)
    run_case(z, d, [-1] + [int(rng.integers(max(0, u - 9), u)) for u in range(1, 256)])


def test_other_stream_and_graph():
    torch, dev = torch_dev()
    z, d, parent = make(2, 3, 7000, 30, torch.bfloat16, seed=6, mask_rows=(2, 3))
    want = call(z, d, parent, -1.0)["logits"].clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = call(z, d, parent, -1.0, stream=s)["logits"]
    s.synchronize()
    assert torch.equal(got, want)
    args = (z, i32(d["hist"]), i32(d["hlen"]))
    out = {"logits": torch.empty_like(z)}
    rep = torch.from_numpy(d["rep"]).to(dev)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ssd.process_logits(*args, repetition=rep, out=out)
    z.neg_()
    g.replay()
    assert torch.equal(out["logits"], ssd.process_logits(*args, repetition=rep)["logits"])


def test_masked_rows_verify():
    """Rows masked with MASKED_LOGIT verify: only allowed tokens come out."""
    torch, dev = torch_dev()
    B, K, V = 8, 4, 50000
    gen = torch.Generator(device=dev).manual_seed(1)
    tg = torch.randn((B, K + 1, V), generator=gen, device=dev)
    dg = torch.randn((B, K + 1, V), generator=gen, device=dev)
    ok = np.zeros((B, K + 1, V), bool)
    rng = np.random.default_rng(1)
    for b in range(B):
        ok[b, :, rng.integers(0, V, 20)] = True
    m = torch.from_numpy(pack(ok)).to(dev)
    tg = ssd.process_logits(tg, mask=m)["logits"]
    dg = ssd.process_logits(dg, mask=m)["logits"]
    tok = torch.argmax(dg[:, :K], -1).int()
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    o = ssd.verify(tg, dg, tok, np.arange(B, dtype=np.uint64), 0, [2] * (K + 1), dev_status=status)
    assert int(status.item()) == 0
    k, t = o["accept_len"].cpu().numpy(), o["bonus"].cpu().numpy()
    assert all(ok[b, k[b], t[b]] for b in range(B))
    assert np.isfinite(o["resid_mass"].cpu().numpy()).all()


def test_refusals():
    torch, dev = torch_dev()
    z = torch.zeros((2, 3, 64), device=dev)
    i2 = torch.zeros(2, dtype=torch.int32, device=dev)
    h = torch.zeros((2, 4), dtype=torch.int32, device=dev)
    for kw in (dict(history=h), dict(history=h, history_len=i2.long()),
               dict(history=h[:1], history_len=i2), dict(history=h.t(), history_len=i2),
               dict(repetition=torch.ones(3, device=dev)), dict(repetition=i2),
               dict(draft_tokens=h), dict(bias_ids=h), dict(mask=h),
               dict(mask=torch.zeros((2, 3, 3), dtype=torch.int32, device=dev)),
               dict(mask=torch.zeros((2, 2, 2), dtype=torch.int32, device=dev)),
               dict(fill=float("nan")), dict(parent=[-1, 0]), dict(parent=[-1, 2, 0]),
               dict(out={"logits": z[:1]}), dict(history=h.cpu(), history_len=i2)):
        with pytest.raises(ssd.SSDError):
            ssd.process_logits(z, **kw)
    with pytest.raises(ssd.SSDError):
        ssd.process_logits(z.half())
    with pytest.raises(ssd.SSDError):
        ssd.process_logits(z[0])
