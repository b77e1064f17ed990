#!/usr/bin/env python
"""Rounds of speculative decoding with drafts as a tree, over a paged cache, with a toy model.

The model has a few attention layers whose queries, keys and values are looked up by token; the
drafter is a table of logits by token.  Prompts are read in, and each is continued by several
samples.  A round, for all rows:

  1. saguaro_sample   every node of the tree draws its children from its drafter's logits;
  2. tree_attention   the target's pass over the nodes, layer by layer: each node over the
                      row's cache and the nodes on its path;
  3. tree_verify      accepted paths and bonus tokens;
  4. page_plan        pages and slots of the tokens that stay;
  5. append_path      the accepted nodes' keys and values, of all layers, into those slots.

Before the first round fork_rows makes the samples of the prompts, and between two rounds it ends
some rows and continues others in their place.

    python examples/tree_rounds.py --rounds 4
"""

from __future__ import annotations

import argparse
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import sampling_ssd_verify_gb300 as ssd  # noqa: E402


class Model:
    """Attention layers over a paged cache that it owns; the drafter's logits by token."""

    def __init__(self, V, L=3, Hq=8, Hkv=2, D=64, pages=128, page=16, device="cuda", seed=0):
        g = torch.Generator(device=device).manual_seed(seed)

        def table(*shape, by=1.0):
            return (torch.randn(shape, generator=g, device=device) * by).to(torch.bfloat16)

        self.L, self.page = L, page
        self.q, self.k, self.v = table(L, V, Hq, D), table(L, V, Hkv, D), table(L, V, Hkv, D)
        self.head = table(Hq * D, V, by=4 * (Hq * D) ** -0.5)
        self.drafter = table(V, V, by=2.0)
        self.k_cache = table(L, pages, page, Hkv, D, by=0.0)
        self.v_cache = torch.zeros_like(self.k_cache)

    def nodes(self, tokens):
        """Keys and values of tokens [B, N], of all layers: [L, B, N, Hkv, D]."""
        return self.k[:, tokens.long()], self.v[:, tokens.long()]

    def logits(self, tokens, k, v, rows, parent):
        """The target's logits [B, N, V] after every node."""
        y = 0
        for layer in range(self.L):
            y = y + ssd.tree_attention(self.q[layer][tokens.long()], k[layer], v[layer],
                                       self.k_cache[layer], self.v_cache[layer], rows.tables,
                                       rows.lens, parent=parent)["out"].float()
        return (y.flatten(2).to(torch.bfloat16) @ self.head).contiguous()


class Rows:
    """Block tables over a pool of pages that rows may share."""

    def __init__(self, n, cols, pages, device="cuda"):
        i32 = dict(dtype=torch.int32, device=device)
        self.lens, self.held = torch.zeros(n, **i32), torch.zeros(n, **i32)
        self.tables = torch.full((n, cols), -1, **i32)
        self.shares = torch.zeros(pages, **i32)
        self.free, self.count = torch.arange(pages, **i32), torch.tensor([pages], **i32)

    def append(self, model, k, v, new, path, status):
        """The first new [n] nodes of every row's path join its cache."""
        p = ssd.page_plan(self.lens, new, self.held, self.tables, self.free, self.count, model.page,
                          k.shape[1] * k.shape[2], dev_status=status)
        ssd.append_path(k, v, model.k_cache, model.v_cache, p["slots"], p["owner"], p["cu"], path,
                        dev_status=status)
        self.lens, self.held, self.count = p["kv_len"], p["held"], p["free_count"]

    def fork(self, model, src, status):
        """Row b continues row src[b]; rows that nobody continues end."""
        o = ssd.fork_rows(src, self.lens, self.held, self.tables, self.shares, self.free,
                          self.count, model.page, model.k_cache, model.v_cache, dev_status=status)
        self.lens, self.held, self.tables = o["lens"], o["held"], o["tables"]
        self.shares, self.count = o["shares"], o["free_count"]


def run(rounds=4, prompts=3, samples=4, V=512, seed=0, device="cuda"):
    """Returns the accepted drafts per round [rounds, B], the rows, the model, every row's tokens
    and the device status."""
    i32 = dict(dtype=torch.int32, device=device)
    rng = np.random.default_rng(seed)
    status = torch.zeros(1, **i32)
    model = Model(V, device=device, seed=seed)
    rows = Rows(prompts, 16, 128, device)
    parent = np.array([-1, 0, 0, 0, 1, 1, 2, 4], dtype=np.int32)
    N, B = len(parent), prompts * samples

    # the prompts: a chain each, all but its last token into the cache
    n = rng.integers(5, 40, prompts)
    text = [rng.integers(0, V, k).tolist() for k in n]
    tokens = torch.zeros((prompts, 40), **i32)
    for b, t in enumerate(text):
        tokens[b, :len(t)] = torch.tensor(t, **i32)
    k, v = model.nodes(tokens)
    rows.append(model, k, v, torch.from_numpy((n - 1).astype(np.int32)).to(device), None, status)

    # their samples
    src = np.repeat(np.arange(prompts), samples)
    rows.fork(model, torch.from_numpy(src.astype(np.int32)).to(device), status)
    text = [list(text[s]) for s in src]
    last = torch.tensor([t[-1] for t in text], **i32)
    seeds = torch.from_numpy(rng.integers(1, 1 << 60, B).astype(np.int64)).to(device)

    accepted = []
    for rnd in range(rounds):
        tokens = torch.zeros((B, N), **i32)
        tokens[:, 0] = last
        for u in range(1, N):
            z = model.drafter[tokens[:, parent[u]].long()]
            tokens[:, u] = ssd.saguaro_sample(z, 1.0, 1.0, 1, seeds, u, rnd,
                                              dev_status=status)["token"]
        draft = model.drafter[tokens.long()]
        k, v = model.nodes(tokens)
        # the drafter has its say in the target, so that some drafts are accepted
        target = model.logits(tokens, k, v, rows, parent) + draft
        o = ssd.tree_verify(target, draft, parent, tokens, seeds, rnd, 1.0, dev_status=status)
        path = o["path"]
        rows.append(model, k, v, o["accept_len"] + 1, path, status)
        last = o["bonus"]
        accepted.append(o["accept_len"].cpu())
        for b, (p, t) in enumerate(zip(path.tolist(), last.tolist())):
            text[b] += [int(tokens[b, u]) for u in p[:int(accepted[-1][b])]] + [t]

        if rnd + 1 < rounds:  # the first row ends, the last one goes on twice
            src = np.concatenate([[B - 1], np.arange(1, B)])
            rows.fork(model, torch.from_numpy(src.astype(np.int32)).to(device), status)
            text = [list(text[s]) for s in src]
            last = last[torch.from_numpy(src).to(device)]
            seeds = torch.cat([seeds[-1:] + 1 + rnd, seeds[1:]])
    return torch.stack(accepted), rows, model, text, int(status.item())


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--rounds", type=int, default=4)
    ap.add_argument("--prompts", type=int, default=3)
    ap.add_argument("--samples", type=int, default=4)
    a = ap.parse_args()
    ssd.build()
    accepted, rows, model, text, status = run(a.rounds, a.prompts, a.samples)
    print("accepted drafts per round:", accepted.tolist(), "status:", status)
    for b, t in enumerate(text):
        print(f"row {b}: {len(t)} tokens, pages {rows.tables[b, :int(rows.held[b])].tolist()}")


if __name__ == "__main__":
    main()
