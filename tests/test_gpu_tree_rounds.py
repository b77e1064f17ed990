"""The operators around tree verification together: a few rounds of the example leave the caches,
pages and tokens that a loop over plain lists does."""

import importlib.util
import os

import numpy as np
import pytest

import sampling_ssd_verify_gb300 as ssd
from tests.parity import torch_dev

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    ssd.build()
    spec = importlib.util.spec_from_file_location("tree_rounds",
                                                  os.path.join(ROOT, "examples", "tree_rounds.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("seed", [0, 1, 2])
def test_rounds(example, seed):
    torch, dev = torch_dev()
    accepted, rows, model, text, status = example.run(rounds=5, seed=seed)
    assert status == 0
    assert int(accepted.min()) >= 0 and int(accepted.max()) > 0
    B, page = len(text), model.page
    lens, held, tables = (x.cpu().numpy() for x in (rows.lens, rows.held, rows.tables))
    # a row's cache holds all of its tokens but the last, in every layer
    for b, t in enumerate(text):
        assert lens[b] == len(t) - 1 and held[b] >= -(-lens[b] // page)
        at = np.arange(lens[b])
        pages, off = torch.from_numpy(tables[b, at // page]).to(dev).long(), \
            torch.from_numpy(at % page).to(dev)
        tokens = torch.tensor(t[:-1], device=dev)
        assert torch.equal(model.k_cache[:, pages, off], model.k[:, tokens])
        assert torch.equal(model.v_cache[:, pages, off], model.v[:, tokens])
    # every page is free, or held by as many rows as shares says
    holders = np.bincount(np.concatenate([tables[b, :held[b]] for b in range(B)]),
                          minlength=rows.shares.numel())
    free = rows.free[:int(rows.count)].cpu().numpy()
    assert len(set(free.tolist())) == len(free)
    assert (holders[free] == 0).all() and len(free) + (holders > 0).sum() == len(holders)
    np.testing.assert_array_equal(rows.shares.cpu().numpy(), np.maximum(holders - 1, 0))
    assert (holders > 1).any()      # the samples of a prompt share its full pages
    # the same again
    again = example.run(rounds=5, seed=seed)
    assert torch.equal(accepted, again[0]) and text == again[3]


def test_logits_do_not_depend_on_how_tokens_came_into_the_cache(example):
    """A node's logits after its tokens were forked, drafted and appended are those of one chain
    over the same tokens: both within the attention's rounding of the definition."""
    torch, dev = torch_dev()
    _, rows, model, text, _ = example.run(rounds=3, seed=4)
    b = len(text) - 1
    t = torch.tensor([text[b]], dtype=torch.int32, device=dev)
    k, v = model.nodes(t)
    one = example.Rows(1, 16, 128, dev)
    whole = [ssd.tree_attention(model.q[l][t.long()], k[l], v[l], model.k_cache[l],
                                model.v_cache[l], one.tables, one.lens) for l in range(model.L)]
    last = t[:, -1:]
    kl, vl = model.nodes(last)
    n = t.shape[1]
    for l in range(model.L):
        got = ssd.tree_attention(model.q[l][last.long()], kl[l], vl[l], model.k_cache[l],
                                 model.v_cache[l], rows.tables[b:b + 1], rows.lens[b:b + 1])
        # as in the operator's own test: weights rounded to bfloat16, sums of n terms; for each
        want = whole[l]["out"][:, -1].double()
        A = v[l].double().abs().amax(1).repeat_interleave(4, 1)    # no output is larger
        S = (model.q[l][last.long()].double().abs().sum(-1).amax() *
             k[l].double().abs().amax() * 64 ** -0.5)
        rs = (64 + 4) * 2.0 ** -23 * S + 2.0 ** -21
        tol = A * (2.0 ** -8 + 2 * rs + (n + 8) * 2.0 ** -23) + 2.0 ** -8 * want.abs()
        assert bool(((got["out"][:, 0].double() - want).abs() <= 2 * tol).all())
        lse = whole[l]["lse"][:, -1].double()
        err = (got["lse"][:, 0].double() - lse).abs()
        assert bool((err <= 2 * (rs + n * 2.0 ** -24 + 2.0 ** -21 + 2.0 ** -23 * lse.abs())).all())
