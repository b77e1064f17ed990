"""How process_logits, page_plan and prefix_attention are called: in inference mode, from
several threads, with the dict of another call, with tables of no columns."""

import ctypes
import threading

import numpy as np
import pytest

import sampling_ssd_verify_gb300 as ssd
from tests import test_gpu_attention as attention
from tests import test_gpu_logits as logits
from tests import test_gpu_pages as pages
from tests.parity import i32, torch_dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    ssd.build()
    ssd.lib()


def test_no_own_tables_whatever_their_columns():
    """NULL tables and lens: no own tokens, whatever `cols` says."""
    torch, dev = torch_dev()
    s = attention.make([3, 2], [50, 7], [0] * 5, 4, 2, 64, 16, torch.bfloat16, own=False)
    want = attention.call(s)
    L = ssd.lib()
    q, k, v = s["q"], s["k"], s["v"]
    for cols in (2, 1000):
        out, lse = torch.full_like(q, 7), torch.empty((5, 4), device=dev)
        a = ssd._Attention(
            0, 5, 4, 2, 64, 2, k.shape[0], 16, q.data_ptr(), q.stride(0), q.stride(1),
            (k.data_ptr(), *k.stride()[:3]), (v.data_ptr(), *v.stride()[:3]), s["pt"].data_ptr(),
            s["pl"].data_ptr(), s["off"].data_ptr(), None, None, s["pt"].stride(0), cols,
            s["pt"].shape[1], cols, out.data_ptr(), out.stride(0), out.stride(1), lse.data_ptr(),
            64 ** -0.5, 0)
        n = L.ssd_prefix_attention_workspace_size(ctypes.byref(a))
        ws = torch.empty(n, dtype=torch.uint8, device=dev)
        st = L.ssd_prefix_attention(ctypes.byref(a), ws.data_ptr(), n, None,
                                    torch.cuda.current_stream().cuda_stream)
        assert st == 0
        assert torch.equal(out, want["out"]) and torch.equal(lse, want["lse"])


@pytest.mark.parametrize("room", [0, 60])
def test_inference_mode(room):
    """A serving program's mode, in which views have no base: outputs new and used again."""
    torch, dev = torch_dev()
    rng = np.random.default_rng(2)
    state = list(pages.random_state(rng, 9, 16, 90, 5, 40, 60))
    state[-1] = room
    with torch.inference_mode():
        pages.run(*state)                 # three calls, two of them with out=
        z, d, parent = logits.make(2, 3, 500, 9, torch.float32, seed=1)
        o = logits.run_case(z, d, parent)
        logits.run_case(z, d, parent, out=o)
        s = attention.make([2, 3], [40, 7], [3] * 5, 4, 2, 64, 16, torch.bfloat16)
        o = attention.call(s)
        attention.check(s, attention.call(s, out=o))


def test_plan_outputs_that_are_not_an_earlier_calls():
    torch, dev = torch_dev()
    i = torch.zeros(4, dtype=torch.int32, device=dev)
    args = (i, i, i, torch.zeros((4, 5), dtype=torch.int32, device=dev), i, i[:1], 16, 8)
    o = ssd.page_plan(*args)
    for out in ({"slots": o["slots"]}, {k: v for k, v in o.items() if k != "served"},
                dict(o, cu=o["cu"].long()), dict(o, cu=o["cu"].cpu()),
                {k: v.clone() for k, v in o.items()}):
        with pytest.raises(ssd.SSDError):
            ssd.page_plan(*args, out=out)
    with torch.inference_mode():
        ssd.page_plan(*args, out=o)       # made outside, used inside


def _hammer(monkeypatch, calls, workers=3, times=3000):
    """Repeats the library calls that `calls` make, each from several threads at once and on
    a stream of its own, with nothing of Python between; returns their status codes."""
    torch, dev = torch_dev()
    L = ssd.lib()
    made = []

    class Record:
        def __getattr__(self, name):
            def call(*args):
                made.append((getattr(L, name), args))
                return made[-1][0](*args)
            return call

    with monkeypatch.context() as m:
        m.setattr(ssd, "_lib", Record())
        for call in calls:
            for _ in range(workers):
                with torch.cuda.stream(torch.cuda.Stream()):
                    call()
    torch.cuda.synchronize()
    seen, start = set(), threading.Barrier(len(made))

    def work(fn, args):
        start.wait()
        for _ in range(times):
            seen.add(fn(*args))

    threads = [threading.Thread(target=work, args=x) for x in made]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    return seen


@pytest.mark.parametrize("dt,sizes", [("float32", (9, 5)), ("bfloat16", (16, 9))])
def test_logits_of_two_sizes_in_several_threads(monkeypatch, dt, sizes):
    """Calls that ask for more shared memory beside calls that ask for less."""
    torch, dev = torch_dev()
    calls, kept = [], []
    for N in sizes:
        z, d, parent = logits.make(310, N, 4099, 9, getattr(torch, dt), seed=N, mask_rows=(1, 1))
        f = lambda a: torch.from_numpy(a).to(dev)  # noqa: E731
        args = (z, i32(d["hist"]), i32(d["hlen"]), i32(d["plen"]))
        kw = dict(draft_tokens=i32(d["drafts"]), parent=parent, repetition=f(d["rep"]),
                  bias_ids=i32(d["ids"]), bias=f(d["bias"]), mask=f(logits.pack(d["mask"])))
        want = ssd.process_logits(*args, **kw)["logits"]

        def call(args=args, kw=kw, want=want):
            kept.append((ssd.process_logits(*args, **kw)["logits"], want))

        calls.append(call)
    torch.cuda.synchronize()
    assert _hammer(monkeypatch, calls) == {0}
    for got, want in kept:
        assert torch.equal(got, want)


def test_plans_of_two_sizes_in_several_threads(monkeypatch):
    torch, dev = torch_dev()
    calls, kept = [], []
    for B in (8000, 2500):
        i = i32(np.full(B, 3))
        args = (i, i, i32(np.ones(B)), i32(np.arange(2 * B).reshape(B, 2)), i32(np.zeros(4)),
                i32([0]), 16, 3 * B)
        want = ssd.page_plan(*args)

        def call(args=args, want=want):
            kept.append((ssd.page_plan(*args), want))

        calls.append(call)
    torch.cuda.synchronize()
    assert _hammer(monkeypatch, calls) == {0}
    for got, want in kept:
        for k in want:
            assert torch.equal(got[k], want[k]), k


@pytest.mark.parametrize("page", [16, 20])
def test_tables_without_columns(page):
    """No prefix in the whole batch, no own page, neither."""
    torch, dev = torch_dev()
    none = torch.empty((2, 0), dtype=torch.int32, device=dev)
    s = attention.make([2, 1], [0, 0], [3, 0, 40], 4, 2, 64, page, torch.bfloat16)
    attention.check(s, attention.call(dict(s, pt=none)))
    attention.check(s, attention.call(dict(s, pt=none, t=s["t"][:, :40 // page + 1].contiguous())))
    rows = torch.empty((3, 0), dtype=torch.int32, device=dev)
    s = attention.make([2, 1], [50, 200], [0, 0, 0], 4, 2, 64, page, torch.bfloat16)
    attention.check(s, attention.call(dict(s, t=rows)))
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    o = attention.call(dict(s, t=rows, pt=none, l=i32([0, 0, 0]), pl=i32([0, 0])),
                       dev_status=status)
    assert bool((o["out"] == 0).all()) and bool((o["lse"] == -float("inf")).all())
    assert int(status.item()) == 0
    attention.call(dict(s, t=rows, l=i32([0, 2, 0])), dev_status=status)
    assert int(status.item()) == ssd.DEV_BAD_LENGTH


def _attn(**kw):
    torch, dev = torch_dev()
    return attention.make([2, 1], [40, 7], [3, 0, 9], 4, 2, 64, 16, torch.bfloat16, **kw)


def test_out_without_lse():
    torch, dev = torch_dev()
    s = _attn()
    y = torch.empty_like(s["q"])
    o = attention.call(s, out={"out": y})
    assert o["out"] is y
    attention.check(s, o)
    first = attention.call(s, lse=False)
    attention.check(s, attention.call(s, out=first))


def test_results_that_were_not_asked_for_are_not_returned():
    """The caller's dict keeps its tensors; the one returned has this call's results alone."""
    torch, dev = torch_dev()
    s = _attn()
    kept = attention.call(s)
    o = attention.call(s, lse=False, out=kept)
    assert "lse" not in o and "lse" in kept and o["out"] is kept["out"]
    assert o["workspace"] is kept["workspace"]
    z = torch.zeros((2, 3, 64), device=dev)
    kept = ssd.process_logits(z, allowed=True)
    o = ssd.process_logits(z, out=kept)
    assert "allowed" not in o and "allowed" in kept and o["logits"] is kept["logits"]


def test_workspace_of_an_earlier_call_grows():
    """The same rows over more groups, more columns, longer own caches."""
    torch, dev = torch_dev()
    small = attention.make([64], [20], [1] * 64, 8, 2, 128, 16, torch.bfloat16)
    o = attention.call(small)
    few = o["workspace"].numel()
    for sizes, pre, suf in (([1] * 64, [200] * 64, [5] * 64), ([64], [900], [2000] + [3] * 63)):
        s = attention.make(sizes, pre, suf, 8, 2, 128, 16, torch.bfloat16)
        attention.check(s, attention.call(s, out=o), rows=range(0, 64, 5))
    assert o["workspace"].numel() > few
    attention.check(small, attention.call(small, out=o), rows=range(0, 64, 9))
    with pytest.raises(ssd.SSDError):     # the caller's own is not replaced
        attention.call(s, workspace=torch.empty(few, dtype=torch.uint8, device=dev))


@pytest.mark.parametrize("ask,flag,left", [
    (3, 0, 3),                       # what does not fit the array is taken again
    (1, ssd.DEV_BAD_LENGTH, 4),      # one page of five does not fit
    (9, ssd.DEV_NO_PAGES | ssd.DEV_BAD_LENGTH, 4),  # all six stay: two do not fit
])
def test_surplus_pages_are_flagged_where_they_are_lost(ask, flag, left):
    torch, dev = torch_dev()
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    tables = np.full((2, 10), -1)
    tables[0, :4], tables[1, 0] = [10, 11, 12, 13], 14
    t, free = i32(tables), i32([20, 21, 22, -1])
    # request 0 keeps one page of four, request 1 wants `ask` more
    o = ssd.page_plan(i32([16, 16]), i32([0, 16 * ask]), i32([4, 1]), t, free, i32([3]), 16, 200,
                      dev_status=status)
    assert int(status.item()) == flag
    assert int(o["free_count"].item()) == left
    stack = [20, 21, 22, 11, 12, 13]
    took = stack[::-1][:ask] if ask <= 6 else []
    assert t[1, 1:1 + len(took)].tolist() == took
    assert free.tolist()[:left] == stack[:left]
    assert o["held"].tolist() == [1, 1 + len(took)]


@pytest.mark.parametrize("dt", ["bfloat16", "float32"])
def test_repetition_is_a_quotient(dt):
    """z / r and z * r, each rounded to float32 once and then to the type: equal to the
    last bit, down to the smallest and up to the largest r."""
    torch, dev = torch_dev()
    r = torch.tensor([1.1, 1.3, 0.7, 7.0, 1e-39, 2.0 ** -149, 2.0 ** -127, 3e-38, 1e38, 3.4e38, 2.0 ** 126],
                     dtype=torch.float32)
    B, V = len(r), 3000
    gen = torch.Generator().manual_seed(4)
    z = torch.randn((B, 1, V), generator=gen) * 4
    z[:, :, ::7] *= 1e-38
    z[:, :, 1::7] *= 1e30
    z[:, :, 2] = 0.0
    z = z.to(getattr(torch, dt))
    history = torch.arange(0, V, 2, dtype=torch.int32).repeat(B, 1)
    f = z.float()
    want = f.clone()
    rr = r[:, None, None]
    want[..., ::2] = torch.where(f > 0, f / rr, f * rr)[..., ::2]
    got = ssd.process_logits(z.to(dev), history.to(dev), i32(np.full(B, V // 2)),
                             repetition=r.to(dev))["logits"]
    assert torch.equal(got.cpu(), want.to(z.dtype))


@pytest.mark.parametrize("Hkv,M,R,D", [(8, 1, 1300, 128), (8, 2, 700, 64), (8, 4, 330, 128),
                                       (5, 3, 520, 256), (4, 4, 9, 128)])
@pytest.mark.parametrize("suf", [6, 40])
def test_attention_in_place(Hkv, M, R, D, suf):
    """Outputs over the queries, with values that are no numbers among the own tokens."""
    torch, dev = torch_dev()
    s = attention.make([R], [70], [suf] * R, Hkv * M, Hkv, D, 16, torch.bfloat16, seed=R)
    if suf <= 16:
        s["t"] = s["t"][:, :1].contiguous()   # the join reads them
    s["v"][int(s["t"][R // 2, 0]), 3, 1] = float("nan")
    want = attention.call(s)
    q = s["q"].clone()
    o = attention.call(dict(s, q=q), out={"out": q, "lse": torch.empty_like(want["lse"])})
    assert o["out"] is q
    assert torch.equal(q.view(torch.int16), want["out"].view(torch.int16))
    assert torch.equal(o["lse"], want["lse"])
