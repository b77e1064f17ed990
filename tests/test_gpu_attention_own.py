"""prefix_attention with own caches that are few tokens: those that the join reads itself
(up to 16 tokens, or one page of up to 64), with one or several key/value heads to a warp,
and the same rows with wider tables, whose own tokens go through a kernel of their own."""

import numpy as np
import pytest

import sampling_ssd_verify_gb300 as ssd
from tests import test_gpu_attention as attention
from tests.parity import torch_dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    ssd.build()
    ssd.lib()


def make(sizes, pre, suf, cols, *args, **kw):
    """attention.make with own tables of `cols` columns."""
    s = attention.make(sizes, pre, suf, *args, **kw)
    torch, dev = torch_dev()
    wide = torch.full((len(suf), cols), -12345, dtype=torch.int32, device=dev)
    n = min(cols, s["t"].shape[1])
    wide[:, :n] = s["t"][:, :n]
    return dict(s, t=wide)


def some(R, n=40):
    return sorted({int(r) for r in np.linspace(0, R - 1, n)})


# (key/value heads, query heads to one, rows): how many of them a warp takes goes by the
# rows; with D = 256 half as many rows are enough
PACKS = [
    (8, 1, 1300),    # eight
    (8, 2, 700),     # four
    (6, 2, 900),     # four, then the last two
    (8, 4, 330),     # two
    (5, 3, 520),     # two, then the last one
    (2, 9, 20),      # several warps for a head's query heads
    (4, 4, 9),       # several warps for a row's partials
]


@pytest.mark.parametrize("D,dt", [(64, "bfloat16"), (128, "bfloat16"), (128, "float16"), (256, "bfloat16")])
@pytest.mark.parametrize("Hkv,M,R", PACKS)
@pytest.mark.parametrize("page,cols,most", [
    (16, 1, 16), (64, 1, 64), (48, 1, 41),     # one page: one, two and eight turns
    (8, 2, 16), (5, 3, 15), (1, 16, 16),       # several pages
])
def test_own_tokens_in_the_join(D, dt, Hkv, M, R, page, cols, most):
    torch, dev = torch_dev()
    third = R // 3
    rng = np.random.default_rng(R + page)
    suf = rng.permutation(np.linspace(0, most, R).round().astype(int))
    s = make([third, R - 2 * third, third], [70, 0, 130], suf, cols, Hkv * M, Hkv, D, page,
             attention.dtype_of(dt), seed=R + D)
    attention.poison(s)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    attention.check(s, attention.call(s, dev_status=status), rows=some(R))
    assert int(status.item()) == 0


@pytest.mark.parametrize("Hkv,M,R", PACKS)
def test_own_tokens_alone_in_the_join(Hkv, M, R):
    s = make([R], [0], np.arange(R) * 7 % 15, 2, Hkv * M, Hkv, 128, 7, attention.dtype_of("float16"), seed=R)
    attention.poison(s)
    attention.check(s, attention.call(s), rows=some(R))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("Hkv,M,R", PACKS)
@pytest.mark.parametrize("page,cols,suf", [(16, 1, 6), (64, 1, 41), (8, 2, 13)])
def test_infinite_values_in_the_join(D, Hkv, M, R, page, cols, suf):
    """What no number is in one head's values reaches the rows and query heads that read it,
    to the last bit no others."""
    torch, dev = torch_dev()
    s = make([R // 2, R - R // 2], [70, 33], [suf] * R, cols, Hkv * M, Hkv, D, page, torch.float16, seed=R)
    want = attention.call(s)["out"].clone()
    hit = torch.zeros((R, Hkv * M), dtype=torch.bool, device=dev)
    v = s["v"]
    for r, h, x in ((0, 1, float("inf")), (R - 1, 0, float("nan")), (R // 3, Hkv - 1, float("-inf")),
                    (R // 3 + 1, Hkv // 2, float("nan"))):
        v[int(s["t"][r, (suf - 1) // page]), (suf - 1) % page, h] = x
        hit[r, h * M:(h + 1) * M] = True
    got = attention.call(s)["out"]
    assert torch.equal(got[~hit], want[~hit])
    assert bool(torch.isfinite(got[~hit]).all()) and not bool(torch.isfinite(got[hit]).any())


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("Hkv,M,R", PACKS)
def test_queries_that_are_no_numbers_in_the_join(D, Hkv, M, R):
    torch, dev = torch_dev()
    s = make([R], [100], [6] * R, 1, Hkv * M, Hkv, D, 16, torch.bfloat16, seed=R)
    want = attention.call(s)["out"].clone()
    s["q"][3, 1] = float("nan")
    s["q"][R - 2, 0, 7] = float("inf")
    keep = torch.ones((R, Hkv * M), dtype=torch.bool, device=dev)
    keep[3, 1] = keep[R - 2, 0] = False
    got = attention.call(s)["out"]
    assert torch.equal(got[keep], want[keep])
    assert not bool(torch.isfinite(got[~keep]).any())


@pytest.mark.parametrize("dt", attention.DT)
@pytest.mark.parametrize("D,page", [(64, 16), (128, 16), (256, 16), (128, 64), (128, 20)])
def test_few_own_tokens_in_tables_of_any_width(dt, D, page):
    """The same rows with tables as narrow as they go and as a pool's fixed width."""
    suf = [1, 2, 3, 4, 0, 9, 16, 5] * 40
    for cols in (1, 2, 4, 64):
        s = make([8] * 40, [90] * 40, suf, cols, 16, 4, D, page, attention.dtype_of(dt), seed=D)
        attention.poison(s)
        attention.check(s, attention.call(s), rows=some(320, 24))


@pytest.mark.parametrize("page,cols,bad", [(16, 1, 0), (8, 2, 1)])
def test_bad_pages_and_lengths_in_the_join(page, cols, bad):
    torch, dev = torch_dev()
    R = 700
    s = make([R], [50], [16] * R, cols, 16, 8, 128, page, torch.bfloat16, seed=page)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    want = attention.call(s, dev_status=status)
    assert int(status.item()) == 0
    others = torch.arange(R, device=dev) != 5
    free = [p for p in range(s["k"].shape[0])
            if p not in s["pt"][0].tolist() and p not in s["t"].flatten().tolist()][0]
    s["k"][free], s["v"][free] = 0, 0
    zeros = s["t"].clone()
    zeros[5, bad] = free
    zeros = attention.call(dict(s, t=zeros))
    for x in (-1, s["k"].shape[0], 2 ** 31 - 1):
        t = s["t"].clone()
        t[5, bad] = x
        status.zero_()
        got = attention.call(dict(s, t=t), dev_status=status)
        assert int(status.item()) == ssd.DEV_BAD_PAGE
        assert torch.equal(got["out"][others], want["out"][others])
        assert torch.equal(got["out"], zeros["out"]) and torch.equal(got["lse"], zeros["lse"])
    for n in (-1, 17, 2 ** 31 - 1):
        l = s["l"].clone()
        l[5] = n
        status.zero_()
        got = attention.call(dict(s, l=l), dev_status=status)
        assert int(status.item()) == ssd.DEV_BAD_LENGTH
        assert torch.equal(got["out"][others], want["out"][others])


@pytest.mark.parametrize("scale", [0.0, -0.2])
@pytest.mark.parametrize("cols", [1, 3])
def test_scales_that_are_not_positive(scale, cols):
    s = make([20, 3], [300, 129], [9] * 23, cols, 8, 2, 128, 16, attention.dtype_of("bfloat16"))
    attention.poison(s)
    attention.check(s, attention.call(s, scale=scale), scale=scale)
