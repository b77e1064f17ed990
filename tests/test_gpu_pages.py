"""page_plan against a plain simulation, request by request, with a Python
list for the stack of free pages.  Whole numbers: everything is equal."""

import numpy as np
import pytest

import sampling_ssd_verify_gb300 as ssd
from tests.parity import i32, torch_dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    ssd.build()
    ssd.lib()


def simulate(lens, new, held, tables, free, count, page, rows):
    tables, cap, cols = [list(map(int, t)) for t in tables], len(free), tables.shape[1]
    n = min(max(count, 0), cap)
    bad = ssd.DEV_BAD_LENGTH if n != count else 0
    stack = list(map(int, free[:n]))
    ok, need = [], []
    for b, (l, k, h) in enumerate(zip(lens, new, held)):
        good = l >= 0 and k >= 0 and 0 <= h <= cols and l + k <= cols * page and l <= h * page
        need.append(-(-(l + k) // page) if good else h)
        ok.append(good)
        if not good:
            bad |= ssd.DEV_BAD_LENGTH
        elif need[b] < h:
            stack += tables[b][need[b]:h]
    if len(stack) > cap:
        bad |= ssd.DEV_BAD_LENGTH
    after = stack[:cap] + list(map(int, free[len(stack):]))
    o = dict(slots=[], positions=[], owner=[], cu=[0], kv_len=[], held=[], served=[])
    gone = False
    for b, (l, k, h) in enumerate(zip(lens, new, held)):
        if not ok[b]:  # inconsistent: no rows
            k = 0
        if ok[b] and need[b] > h:
            gone = gone or need[b] - h > len(stack)
            if gone:
                ok[b] = False
                bad |= ssd.DEV_NO_PAGES
            else:
                for c in range(h, need[b]):
                    tables[b][c] = stack.pop()
        for i in range(k):
            p = l + i
            o["slots"].append(tables[b][p // page] * page + p % page if ok[b] else -1)
            o["positions"].append(p)
            o["owner"].append(b)
        o["cu"].append(o["cu"][-1] + k)
        o["kv_len"].append(l + k if ok[b] else l)
        o["held"].append(need[b] if ok[b] else h)
        o["served"].append(int(ok[b]))
    if o["cu"][-1] > rows:
        bad |= ssd.DEV_BAD_LENGTH
    for name in ("slots", "positions", "owner"):
        o[name] = (o[name] + [-1] * rows)[:rows]
    return dict(o, free_count=[min(len(stack), cap)], tables=tables, free_pages=after), bad


def run(lens, new, held, tables, free, count, page, rows, **kw):
    torch, dev = torch_dev()
    want, bad = simulate(lens, new, held, tables, free, count, page, rows)
    t, f = i32(tables), i32(free)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    args = (i32(lens), i32(new), i32(held), t, f, i32([count]), page, rows)
    o = ssd.page_plan(*args, dev_status=status, **kw)
    torch.cuda.synchronize()
    for again in range(2):  # a call repeated on the same inputs gives the same
        got = dict(o, tables=t, free_pages=f)
        for k, v in want.items():
            np.testing.assert_array_equal(got[k].cpu().numpy(), np.asarray(v), err_msg=k)
        assert int(status.item()) == bad
        o = ssd.page_plan(*args, dev_status=status, out=o)
    return o


def random_state(rng, B, page, most, new_hi, spare, free):
    lens = rng.integers(0, most + 1, B)
    new = rng.integers(0, new_hi + 1, B)
    held = -(-(lens + rng.integers(0, spare + 1, B)) // page)
    cols = -(-(most + max(spare, new_hi)) // page) + 1
    ids = rng.permutation(int(held.sum()) + free)
    tables = np.full((B, cols), -1)
    tables[np.arange(cols) < held[:, None]] = ids[free:]
    back = np.maximum(held - -(-(lens + new) // page), 0).sum()
    stack = np.concatenate([ids[:free], np.full(int(back), -1)])
    return lens, new, held, tables, stack, free, page, int(new.sum())


@pytest.mark.parametrize("B,page,most,new_hi,spare,free", [
    (1, 16, 0, 1, 0, 3), (1, 1, 5, 9, 3, 40), (3, 7, 40, 20, 30, 30), (32, 16, 900, 5, 40, 60),
    (257, 64, 4000, 9, 200, 300), (600, 16, 300, 900, 50, 40000), (513, 20, 60, 700, 0, 5000),
    (8192, 128, 1000, 3, 300, 9000), (5, 16, 100, 0, 64, 0), (40, 8, 100, 30, 100, 25),
])
def test_matches_simulation(B, page, most, new_hi, spare, free):
    rng = np.random.default_rng(B + page)
    run(*random_state(rng, B, page, most, new_hi, spare, free))


def test_page_ids_past_32_bits_of_slots():
    rng = np.random.default_rng(0)
    lens, new, held, tables, stack, free, page, rows = random_state(rng, 20, 128, 500, 9, 10, 90)
    big = 2 ** 31 - 1 - 4000
    tables = np.where(tables >= 0, tables + big, tables)
    run(lens, new, held, tables, np.where(stack >= 0, stack + big, stack), free, page, rows)


@pytest.mark.parametrize("room", [0, 1, 50, 100000])
def test_rows_of_any_number(room):
    rng = np.random.default_rng(4)
    s = list(random_state(rng, 30, 16, 200, 12, 20, 100))
    s[-1] = room
    run(*s)


def test_inconsistent_lengths_are_refused_one_by_one():
    rng = np.random.default_rng(7)
    lens, new, held, tables, stack, free, page, rows = random_state(rng, 12, 16, 200, 40, 30, 200)
    cols = tables.shape[1]
    lens[0], new[1], held[2] = -1, -4, -1
    held[3] = cols + 1
    new[4] = cols * page + 1
    lens[5], held[5] = 100, 2
    lens[6], new[6] = 2 ** 31 - 1, 2 ** 31 - 1
    run(lens, new, held, tables, stack, free, page, 500)


@pytest.mark.parametrize("count", [-3, 10 ** 6])
def test_bad_count_of_free_pages(count):
    rng = np.random.default_rng(9)
    lens, new, held, tables, stack, free, page, rows = random_state(rng, 9, 16, 200, 40, 0, 200)
    run(lens, new, held, tables, stack, count, page, rows)


def test_returned_pages_past_the_array_are_flagged():
    rng = np.random.default_rng(11)
    lens, new, held, tables, stack, free, page, rows = random_state(rng, 9, 16, 300, 0, 200, 5)
    run(lens, new, held, tables, stack[:8], free, page, rows)


def test_rounds_follow_one_another():
    """Lengths that grow by what was accepted: pages are never held twice."""
    torch, dev = torch_dev()
    rng = np.random.default_rng(3)
    B, page, total, cols = 24, 8, 700, 40
    lens = i32(np.zeros(B))
    held, count = i32(np.zeros(B)), i32([total])
    tables, free = i32(np.full((B, cols), -1)), i32(rng.permutation(total))
    for step in range(12):
        new = i32(rng.integers(0, 20, B))
        o = ssd.page_plan(lens, new, held, tables, free, count, page, 20 * B)
        h, n = o["held"].cpu().numpy(), int(o["free_count"].item())
        t = tables.cpu().numpy()
        mine = np.concatenate([t[b, :h[b]] for b in range(B)] + [free.cpu().numpy()[:n]])
        assert sorted(mine) == list(range(total))
        s = o["slots"].cpu().numpy()
        s = s[s >= 0]
        assert len(set(s)) == len(s) == int(new.sum().item())
        keep = torch.minimum(new, i32(rng.integers(0, 20, B)))  # accepted
        lens, held, count = lens + keep, o["held"], o["free_count"]


def test_refusals():
    torch, dev = torch_dev()
    i = torch.zeros(4, dtype=torch.int32, device=dev)
    t = torch.zeros((4, 5), dtype=torch.int32, device=dev)
    ok = (i, i, i, t, i, i[:1], 16, 8)
    o = ssd.page_plan(*ok)
    for out in (dict(o, cu=o["cu"].clone()), dict(o, slots=o["slots"].int()),
                ssd.page_plan(*ok[:-1], 7), ssd.page_plan(i[:3], i[:3], i[:3], t[:3], *ok[4:])):
        with pytest.raises(ssd.SSDError):
            ssd.page_plan(*ok, out=out)
    ssd.page_plan(*ok, out=o)
    for at, x in ((0, i[:3]), (1, i.long()), (2, i.cpu()), (3, t[:3]), (3, t.t()), (3, t.long()),
                  (4, i.float()), (5, i), (6, 0), (7, -1)):
        args = list(ok)
        args[at] = x
        with pytest.raises((ssd.SSDError, RuntimeError)):
            ssd.page_plan(*args)
