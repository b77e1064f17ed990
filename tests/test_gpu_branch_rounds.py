"""The example of a serving loop: it runs, flags nothing, keeps to the grammar, and
the same seed gives the same tokens."""

import importlib.util
import os

import pytest

import sampling_ssd_verify_gb300 as ssd

pytestmark = pytest.mark.gpu


def test_branch_rounds():
    import torch

    ssd.build()
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "branch_rounds.py")
    spec = importlib.util.spec_from_file_location("branch_rounds", path)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    accepted, status, history, lens = ex.run(rounds=4, B=5, seed=3)
    assert status == 0 and accepted.shape == (4, 5)
    assert bool(((accepted >= 0) & (accepted <= 3)).all()) and int(accepted.sum()) > 0
    prompts = lens - accepted.sum(0) - 4
    for b in range(0, 5, 2):  # the grammar of these sequences allows even tokens alone
        assert bool((history[b, prompts[b]:lens[b]] % 2 == 0).all())
    again = ex.run(rounds=4, B=5, seed=3)
    assert torch.equal(accepted, again[0]) and torch.equal(lens, again[3])
    for b in range(5):
        assert torch.equal(history[b, :lens[b]], again[2][b, :lens[b]])
