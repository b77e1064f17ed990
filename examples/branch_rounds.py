#!/usr/bin/env python
"""A few rounds of speculative speculative decoding with a toy drafter, with every
operator of the package where a serving loop has it.

The drafter is one attention layer with random weights over a paged key/value
cache; the target is the drafter's logits with noise, as far as this loop goes.
A round, for all B sequences:

  1. process_logits   repetition penalty, biases and a grammar on the target's and
                      the drafter's rows (row j counts the drafts before it);
  2. verify_round     accepted lengths, bonus tokens, guesses, outcome cache;
  3. page_plan        the pages of the tokens that stay and of the next drafts, and
                      the slots where their keys and values go;
  4. prefix_attention the branches: one row per guess, all rows of a sequence over
                      its prefix, each with its guessed token;
  5. saguaro_sample   the next token of every branch.

    python examples/branch_rounds.py --rounds 4
"""

from __future__ import annotations

import argparse
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import sampling_ssd_verify_gb300 as ssd  # noqa: E402


class Drafter:
    """One attention layer over a paged cache that it owns."""

    def __init__(self, V, Hq=8, Hkv=2, D=64, pages=512, page=16, device="cuda", seed=0):
        g = torch.Generator(device=device).manual_seed(seed)

        def weight(*shape):
            w = torch.randn(shape, generator=g, device=device) / shape[0] ** 0.5
            return w.to(torch.bfloat16)

        self.Hq, self.Hkv, self.D, self.page = Hq, Hkv, D, page
        E = Hq * D
        self.embed, self.head = weight(V, E) * V ** 0.5, weight(E, V)
        self.wq, self.wk, self.wv = weight(E, E), weight(E, Hkv * D), weight(E, Hkv * D)
        self.k = torch.zeros((pages, page, Hkv, D), dtype=torch.bfloat16, device=device)
        self.v = torch.zeros_like(self.k)

    def write(self, tokens, slots):
        """Keys and values of tokens [n] into their slots [n] (negative: nowhere)."""
        x = self.embed[tokens.long()]
        keep = slots >= 0
        for cache, w in ((self.k, self.wk), (self.v, self.wv)):
            cache.view(-1, self.Hkv, self.D)[slots[keep]] = \
                (x @ w).view(-1, self.Hkv, self.D)[keep]

    def logits(self, tokens, *attention):
        """Rows of logits after tokens [R], which are in the cache already."""
        x = self.embed[tokens.long()]
        q = (x @ self.wq).view(-1, self.Hq, self.D)
        y = ssd.prefix_attention(q, self.k, self.v, *attention)["out"]
        return (x + y.reshape(len(x), -1)) @ self.head


class Pages:
    """Block tables of n rows over a pool, and how many tokens and pages each has."""

    def __init__(self, n, cols, free, device="cuda"):
        z = torch.zeros(n, dtype=torch.int32, device=device)
        self.lens, self.held = z, z.clone()
        self.tables = torch.full((n, cols), -1, dtype=torch.int32, device=device)
        self.free = free
        self.count = torch.tensor([len(free)], dtype=torch.int32, device=device)

    def append(self, new, most, page, status):
        """Room for new [n] tokens per row: their slots, row after row."""
        p = ssd.page_plan(self.lens, new, self.held, self.tables, self.free, self.count, page,
                          most, dev_status=status)
        self.held, self.count = p["held"], p["free_count"]
        return p


def run(rounds=3, B=4, K=3, V=2048, F=2, seed=0, device="cuda"):
    """Returns the tokens accepted per round [rounds, B] and the device status."""
    i32 = dict(dtype=torch.int32, device=device)
    gen = torch.Generator(device=device).manual_seed(seed)
    rng = np.random.default_rng(seed)
    status = torch.zeros(1, **i32)
    model = Drafter(V, device=device, seed=seed)
    pool = torch.arange(512, **i32)
    seqs = Pages(B, 32, pool[:256].clone(), device)          # the sequences
    rows = Pages(B * (K + 1) * F, 1, pool[256:].clone(), device)  # their branches
    G = torch.arange(0, B * (K + 1) * F + 1, F, **i32)       # branches of an outcome (b, k)
    one = torch.arange(B + 1, **i32)                          # a row per sequence

    # prompts of 5 to 20 tokens
    n = torch.from_numpy(rng.integers(5, 21, B).astype(np.int32)).to(device)
    history = torch.randint(0, V, (B, 20 + rounds * (K + 1)), generator=gen, **i32)
    p = seqs.append(n, 20 * B, model.page, status)
    used = p["owner"] >= 0
    model.write(history[p["owner"][used].long(), p["positions"][used].long()], p["slots"][used])
    seqs.lens = n
    prompt = n.clone()

    rules = dict(repetition=torch.full((B,), 1.2, device=device),
                 presence=torch.full((B,), 0.1, device=device),
                 frequency=torch.full((B,), 0.05, device=device),
                 bias_ids=torch.randint(0, V, (B, 4), generator=gen, **i32),
                 bias=torch.full((B, 4), -2.0, device=device))
    # the grammar: even tokens for even sequences, anything for the others
    words = torch.full((B, 1, V // 32), -1, **i32)
    words[::2] = 0x55555555
    seeds = torch.from_numpy(rng.integers(1, 1 << 60, B).astype(np.int64)).to(device)
    row_seeds = torch.from_numpy(rng.integers(1, 1 << 60, len(rows.lens)).astype(np.int64)).to(device)
    accepted = []
    for rnd in range(rounds):
        # K drafts and the row after the last, one token at a time; each token's keys
        # and values go to the slots planned for it
        plan = seqs.append(torch.full((B,), K + 1, **i32), B * (K + 1), model.page, status)
        slots = plan["slots"].view(B, K + 1)
        draft = torch.empty((B, K + 1, V), dtype=torch.bfloat16, device=device)
        drafts = torch.zeros((B, K), **i32)
        last = history.gather(1, (seqs.lens - 1)[:, None].long())[:, 0].int()
        for j in range(K + 1):
            z = model.logits(last, seqs.tables, seqs.lens + j, one)
            draft[:, j] = z
            if j < K:
                z = ssd.process_logits(z[:, None], history, seqs.lens + j, prompt, mask=words,
                                       **rules)["logits"]
                last = ssd.saguaro_sample(z[:, 0], 1.0, 1.0, F, seeds, j, rnd,
                                          dev_status=status)["token"]
                drafts[:, j] = last
                history.scatter_(1, (seqs.lens + j)[:, None].long(), last[:, None])
                model.write(last, slots[:, j])
        target = draft.float() + 0.5 * torch.randn(draft.shape, generator=gen, device=device)
        target, draft = (ssd.process_logits(x, history, seqs.lens, prompt, draft_tokens=drafts,
                                            mask=words, dev_status=status, **rules)["logits"]
                         for x in (target.to(torch.bfloat16), draft))
        o = ssd.verify_round(target, draft, drafts, seeds, rnd, [F] * (K + 1), dev_status=status)

        # a branch per guess: its token in a page of its own, its attention over the
        # sequence, the drafts before its position k, and that token
        guesses = o["guesses"].view(-1)
        branch = rows.append(torch.ones_like(rows.lens), len(rows.lens), model.page, status)
        model.write(guesses.clamp(min=0), branch["slots"])
        prefix = (seqs.lens[:, None] + torch.arange(K + 1, **i32)).view(-1)
        z = model.logits(guesses.clamp(min=0), seqs.tables.repeat_interleave(K + 1, 0), prefix, G,
                         rows.tables, branch["kv_len"])
        ssd.saguaro_sample(z, 1.0, 1.0, F, row_seeds, K, rnd, dev_status=status)

        # the accepted drafts and the bonus token join the history
        k = o["accept_len"]
        new = torch.cat([drafts, drafts[:, :1]], 1)
        new.scatter_(1, k[:, None].long(), o["bonus"][:, None])
        model.write(o["bonus"], slots.gather(1, k[:, None].long())[:, 0])
        at = seqs.lens[:, None] + torch.arange(K + 1, **i32)
        stays = torch.arange(K + 1, **i32) <= k[:, None]
        history.scatter_(1, at.long(), torch.where(stays, new, history.gather(1, at.long())))
        seqs.lens = seqs.lens + k + 1
        accepted.append(k)
    return torch.stack(accepted).cpu(), int(status.item()), history.cpu(), seqs.lens.cpu()


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--rounds", type=int, default=3)
    ap.add_argument("--batch", type=int, default=4)
    a = ap.parse_args()
    ssd.build()
    accepted, status, history, lens = run(a.rounds, a.batch)
    print("accepted drafts per round:", accepted.tolist(), "status:", status)
    for b in range(a.batch):
        print(f"sequence {b}:", history[b, :lens[b]].tolist())


if __name__ == "__main__":
    main()
