"""Prompts and two steps with drafted tokens over the latent cache, as a serving loop with speculative decoding would call them.
Random weights, inputs and acceptance; needs a GPU and the built library.

    python examples/draft_step.py [--four-bit]

Prompts: block tables, then the latents normed, rotated and stored.
A step: tables for a request's drafts; their latents normed, rotated to their depth in the tree and stored; the queries normed and rotated;
the drafts attended over the history and their ancestors; then the accepted ones' records moved to the front of the drafts, in every layer's
cache at once, and the pages behind them given back to the pool.
"""
from __future__ import annotations

import argparse
import os
import random
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from sparse_attention_kv_e4m3_gb300 import draft, latent, native  # noqa: E402

LATENT, ROPE, NOPE = 512, 64, 128
SCALE = (NOPE + ROPE) ** -0.5


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Tree:
    """A request's drafts: their parents (-1: the last token of the history), depths and ancestors' bits."""

    def __init__(self, parents):
        self.parents, self.depth, self.seen = parents, [], []
        for j, p in enumerate(parents):
            self.depth.append(self.depth[p] + 1 if p >= 0 else 0)
            self.seen.append((self.seen[p] if p >= 0 else 0) | 1 << j)

    def path_to(self, j):
        path = []
        while j >= 0:
            path.append(j)
            j = self.parents[j]
        return path[::-1]


class Pool:
    """Every layer's cache, one page table, and the requests' state."""

    def __init__(self, layers: int, requests: int, pages_per_request: int, record_format: str, device="cuda"):
        pages = requests * pages_per_request
        self.caches = draft.LayeredCache.empty(layers, pages, ROPE, record_format, device)
        self.page_table = torch.full((requests, pages_per_request), -1, dtype=torch.int32, device=device)
        self.free = torch.randperm(pages, device=device).int()
        self.len = torch.zeros(requests, dtype=torch.int32, device=device)
        self.status = torch.zeros(1, dtype=torch.int32, device=device)
        self.freq = (10000.0 ** (-torch.arange(0, ROPE, 2, dtype=torch.float64, device=device) / ROPE)).float()

    def room(self, new_len: torch.Tensor, n_rows: int) -> latent.StepTables:
        t = latent.csa_build_tables(self.len, new_len, self.page_table, self.free, n_rows, dev_status=self.status)
        self.free = self.free[int(t.taken):]
        return t

    def give_back(self, done: draft.Committed) -> None:
        self.len = done.new_len
        self.free = torch.cat([self.free, done.freed[:int(done.n_freed)]])


def run(prompts=(700, 65, 190, 1), layers: int = 2, heads: int = 16, record_format: str = "bf16", steps: int = 2, seed: int = 0) -> dict:
    gen, rng = torch.Generator(device="cuda").manual_seed(seed), random.Random(seed)

    def rand(*shape):
        return torch.randn(*shape, generator=gen, device="cuda").to(torch.bfloat16)

    n, total = len(prompts), sum(prompts)
    pool = Pool(layers, n, max(prompts) // native.PAGE_RECORDS + 4, record_format)
    weight = [1 + 0.1 * rand(LATENT).float() for _ in range(layers)]
    q_weight = [1 + 0.1 * rand(NOPE + ROPE).float() for _ in range(layers)]
    absorb = [(rand(heads, NOPE, LATENT) * NOPE ** -0.5) for _ in range(layers)]
    # --- the prompts; what each token brings to each layer is kept to look at
    t = pool.room(ints(prompts), total)
    tokens = [rand(total, LATENT + ROPE) for _ in range(layers)]
    for l in range(layers):
        draft.csa_latent_append(tokens[l], t.row_slot, t.row_pos, pool.caches.layers[l], pool.freq, weight=weight[l], dev_status=pool.status)
    pool.len = ints(prompts)
    at = [sum(prompts[:r]) for r in range(n + 1)]
    kept = [[tokens[l][at[r]:at[r + 1]] for r in range(n)] for l in range(layers)]
    done_steps = []
    for _ in range(steps):
        # --- the drafts: a tree a request, its tokens in the order in which they were drafted
        trees = [Tree([rng.randint(max(-1, j - 4), j - 1) for j in range(rng.randint(1, 12))]) for _ in range(n)]
        count = [len(tree.parents) for tree in trees]
        rows = sum(count)
        before, t = pool.len, pool.room(ints(count), rows)
        depth = ints([d for tree in trees for d in tree.depth])
        pos = before[t.row_req.long()] + depth  # a draft's place in its sequence, not in the cache
        mask = torch.tensor([m for tree in trees for m in tree.seen], dtype=torch.int64, device="cuda")[:, None]
        x, seen = [], []
        for l in range(layers):
            cache = pool.caches.layers[l]
            new, q = rand(rows, LATENT + ROPE), rand(rows, heads, NOPE + ROPE)
            draft.csa_latent_append(new, t.row_slot, pos, cache, pool.freq, weight=weight[l], dev_status=pool.status)
            ready, _ = draft.csa_head_norm_rotate(q, pos, pool.freq, q_weight=q_weight[l], dev_status=pool.status)
            absorbed = torch.cat([torch.einsum("bhd,hdc->bhc", ready[..., :NOPE], absorb[l]), ready[..., NOPE:]], -1)
            out, lse = draft.csa_draft_attend(absorbed, cache, pool.page_table, before, t.row_start, scale=SCALE, mask=mask, dev_status=pool.status)
            x.append(new)
            seen.append((q, ready, absorbed, out, lse))
        # --- what the model would have accepted: a path down each tree
        paths = [tree.path_to(rng.randrange(len(tree.parents))) if rng.random() < 0.9 else [] for tree in trees]
        wide = max(1, max(len(p) for p in paths))
        records, table = pool.caches.pages.clone(), pool.page_table.clone()  # as the attention saw them
        done = draft.csa_draft_commit(pool.caches, pool.page_table, before, ints(count), ints([p + [-1] * (wide - len(p)) for p in paths]),
                                      ints([len(p) for p in paths]), dev_status=pool.status)
        pool.give_back(done)
        start = [sum(count[:r]) for r in range(n)]
        for l in range(layers):
            for r in range(n):
                kept[l][r] = torch.cat([kept[l][r], x[l][[start[r] + j for j in paths[r]]]])
        done_steps.append(dict(before=before, trees=trees, tables=t, pos=pos, layers=seen, records=records, table=table, paths=paths, done=done))
    return dict(pool=pool, kept=kept, weight=weight, q_weight=q_weight, steps=done_steps)


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--four-bit", action="store_true", help="hold the latents as MXFP4 records")
    a = ap.parse_args()
    r = run(record_format="mxfp4" if a.four_bit else "bf16")
    torch.cuda.synchronize()
    for s in r["steps"]:
        print("drafts", [len(t.parents) for t in s["trees"]], "| accepted", [len(p) for p in s["paths"]], "| lengths", s["done"].new_len.tolist(),
              "| pages back", int(s["done"].n_freed))
    print("status", int(r["pool"].status))


if __name__ == "__main__":
    main()
