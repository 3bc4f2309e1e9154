"""examples/latent_step.py: the tables, the caches, the indexer and both attentions together."""
import importlib.util
import os

import pytest
import torch

import _latent as L
from conftest import ROOT

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_attention_kv_e4m3_gb300 import build

    build.build()
    spec = importlib.util.spec_from_file_location("latent_step", os.path.join(ROOT, "examples", "latent_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("fmt", ["bf16", "mxfp4"])
def test_prompts_then_a_decode_step(example, fmt):
    prompts = (700, 65, 1300, 1)
    r = example.run(prompts, record_format=fmt, seed=3)
    pool, t = r["pool"], r["tables"]
    assert int(pool.status) == 0
    assert pool.len.tolist() == [n + 1 for n in prompts] and t.row_pos.tolist() == list(prompts)
    cache = pool.latents.pages.reshape(-1, pool.latents.record_bytes)
    values = L.values(cache, fmt, 64)
    start = 0
    for b, n in enumerate(prompts):
        pos = torch.arange(n + 1, device="cuda")
        at = pool.page_table[b].long()[pos // 64] * 64 + pos % 64
        # what the prompt's attention read back is what the cache holds
        assert torch.equal(r["rows"][start:start + n].double(), values[at[:n]].to(torch.bfloat16).double())
        start += n
        # distinct positions of the row, all of them where they are not more than 512
        idx = r["idx"][b][r["idx"][b] >= 0].long()
        assert idx.numel() == min(n + 1, 512) and idx.unique().numel() == idx.numel() and int(idx.max()) <= n
        k = values[at[idx]]
        L.hold(r["attended"][b], r["lse"][b], L.softmax_out(r["absorbed"][b].double(), k, k[:, :512], example.SCALE, 576))


def test_absorbed_and_expanded_forms_agree(example):
    """The last prompt row's expanded attention against the absorbed one over the same records: the two differ by the
    roundings of the expanded keys and values and of the absorbed queries to bf16 (2^-8 relative each, and sums of 512
    of them), far below the 5% that a wrong head, position or scale would exceed."""
    import sparse_attention_kv_e4m3_gb300.latent as latent

    prompts = (700, 65, 1300, 1)
    r = example.run(prompts, seed=4)
    layer, pool = r["layer"], r["pool"]
    last = torch.tensor(prompts, device="cuda").cumsum(0) - 1
    q = layer.absorb(r["q"][last])
    o, _ = latent.csa_latent_attend(q, pool.latents, pool.page_table, torch.tensor(prompts, dtype=torch.int32, device="cuda"),
                                    scale=example.SCALE)
    a, b = layer.values(o).double(), r["prompt_out"][last].double()
    assert ((a - b).norm(dim=(1, 2)) <= 0.05 * b.norm(dim=(1, 2))).all()
