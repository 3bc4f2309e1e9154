"""One prompt wave and one decode step through the indexer and the latent cache, as a serving
loop would call them. Random weights and inputs; needs a GPU and the built library.

    python examples/latent_step.py [--four-bit]

Prompt wave, per layer: block tables from the prompts' lengths; the new latents into the cache and the
index keys into the indexer's cache (one page table for both); the stored latents read back, expanded per head
(one matrix product) and attended causally.
Decode step: tables for one more record a request; its latent and key stored; the indexer's best positions;
absorbed latent attention over those positions.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from sparse_attention_kv_e4m3_gb300 import latent, native  # noqa: E402

LATENT, ROPE, NOPE, VDIM, INDEX_HEADS, INDEX_DIM = 512, 64, 128, 128, 64, 128
SCALE = (NOPE + ROPE) ** -0.5


class Layer:
    """Weights of one layer: the expansion of a latent into a head's keys and values."""

    def __init__(self, heads: int, gen: torch.Generator, device="cuda"):
        def rand(*shape):
            return (torch.randn(*shape, generator=gen, device=device) * shape[-1] ** -0.5).to(torch.bfloat16)

        self.heads = heads
        self.w_k, self.w_v = rand(heads, NOPE, LATENT), rand(heads, VDIM, LATENT)
        self.w_kv = torch.cat([self.w_k, self.w_v], 1).reshape(heads * (NOPE + VDIM), LATENT)

    def expand(self, rows: torch.Tensor):
        """Rows [n, 512 + 64] of the cache -> (k_nope, k_rope, v) of csa_latent_prefill."""
        kv = (rows[:, :LATENT] @ self.w_kv.t()).reshape(rows.shape[0], self.heads, NOPE + VDIM)
        return kv[..., :NOPE], rows[:, LATENT:], kv[..., NOPE:]

    def absorb(self, q: torch.Tensor) -> torch.Tensor:
        """q [n, heads, 192] -> the absorbed queries [n, heads, 512 + 64] of csa_latent_attend."""
        return torch.cat([torch.einsum("bhd,hdc->bhc", q[..., :NOPE], self.w_k), q[..., NOPE:]], -1)

    def values(self, o: torch.Tensor) -> torch.Tensor:
        """The attended latents [n, heads, 512] as the heads' values [n, heads, 128]."""
        return torch.einsum("bhc,hvc->bhv", o, self.w_v)


class Pool:
    """The pages of a layer, shared by the indexer's keys and the latents, and the requests' state."""

    def __init__(self, requests: int, pages_per_request: int, record_format: str, device="cuda"):
        pages = requests * pages_per_request
        self.latents = latent.LatentCache.empty(pages, ROPE, record_format, device)
        self.keys = torch.zeros((pages, native.PAGE_BYTES), dtype=torch.uint8, device=device)
        self.page_table = torch.full((requests, pages_per_request), -1, dtype=torch.int32, device=device)
        self.free = torch.randperm(pages, device=device).int()
        self.len = torch.zeros(requests, dtype=torch.int32, device=device)
        self.status = torch.zeros(1, dtype=torch.int32, device=device)

    def step(self, new_len: torch.Tensor, n_rows: int, latents: torch.Tensor, keys: torch.Tensor) -> latent.StepTables:
        """Room for new_len[r] more records of each request, and those records stored."""
        t = latent.csa_build_tables(self.len, new_len, self.page_table, self.free, n_rows, dev_status=self.status)
        latent.csa_latent_write(latents, t.row_slot, self.latents, dev_status=self.status)
        native.csa_index_write_keys(keys, t.row_pos, self.keys, self.page_table, row_req=t.row_req, dev_status=self.status)
        # a real pool keeps its free list on the device too; here the pages handed out move to its end
        self.free = torch.roll(self.free, -int(t.taken))
        self.len = self.len + new_len
        return t


def run(prompts=(700, 65, 1300, 1), heads: int = 16, top: int = 512, record_format: str = "bf16", seed: int = 0) -> dict:
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def rand(*shape):
        return torch.randn(*shape, generator=gen, device="cuda").to(torch.bfloat16)

    layer, n = Layer(heads, gen), len(prompts)
    pool = Pool(n, max(prompts) // native.PAGE_RECORDS + 2, record_format)
    # --- the prompts
    total = sum(prompts)
    new = torch.tensor(prompts, dtype=torch.int32, device="cuda")
    t = pool.step(new, total, rand(total, LATENT + ROPE), rand(total, INDEX_DIM))
    rows = latent.csa_latent_read(pool.latents, pool.page_table, t.kv_start, total, dev_status=pool.status)
    q = rand(total, heads, NOPE + ROPE)
    k_nope, k_rope, v = layer.expand(rows)
    prompt_out, prompt_lse = latent.csa_latent_prefill(q, k_nope, k_rope, v, t.row_start, t.kv_start, scale=SCALE,
                                                       dev_status=pool.status)
    # --- one decode step
    t = pool.step(torch.ones_like(new), n, rand(n, LATENT + ROPE), rand(n, INDEX_DIM))
    index = native.Problem(q=rand(n, INDEX_HEADS, INDEX_DIM), fused_w=rand(n, INDEX_HEADS).float() * (INDEX_DIM * INDEX_HEADS) ** -0.5,
                           kv=pool.keys, page_table=pool.page_table, q_len=t.row_len, q_req=t.row_req, dev_status=pool.status)
    idx, _ = native.csa_index_score_topk_fused(index, top)
    step_q = rand(n, heads, NOPE + ROPE)
    absorbed = layer.absorb(step_q)
    o, lse = latent.csa_latent_attend(absorbed, pool.latents, pool.page_table, t.row_len, scale=SCALE, idx=idx, row_req=t.row_req,
                                      dev_status=pool.status)
    return dict(layer=layer, pool=pool, rows=rows, q=q, prompt_out=prompt_out, prompt_lse=prompt_lse, tables=t, idx=idx,
                absorbed=absorbed, attended=o, lse=lse, out=layer.values(o))


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--four-bit", action="store_true", help="hold the latents as MXFP4 records")
    a = ap.parse_args()
    r = run(record_format="mxfp4" if a.four_bit else "bf16")
    torch.cuda.synchronize()
    print("status", int(r["pool"].status), "| prompt rows", tuple(r["prompt_out"].shape), "| decode rows", tuple(r["out"].shape),
          "| positions a row", (r["idx"] >= 0).sum(1).tolist())


if __name__ == "__main__":
    main()
