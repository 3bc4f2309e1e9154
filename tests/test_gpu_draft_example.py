"""examples/draft_step.py: tables, the rotating writer, norms and rotation of queries, attention of the drafts and the move of the
accepted ones together, over two steps."""
import importlib.util
import os

import pytest
import torch

import _draft as D
import _latent as L
from conftest import ROOT

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_attention_kv_e4m3_gb300 import build

    build.build()
    spec = importlib.util.spec_from_file_location("draft_step", os.path.join(ROOT, "examples", "draft_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("fmt", ["bf16", "mxfp4"])
def test_prompts_and_two_steps(example, fmt):
    r = example.run(record_format=fmt, seed=5)
    pool, rec = r["pool"], L.record_bytes(fmt, 64)
    assert int(pool.status) == 0
    table, n = pool.page_table.long(), pool.len.shape[0]

    def slots(request, count, table=table):
        pos = torch.arange(count, device="cuda")
        return table[request, pos // 64] * 64 + pos % 64

    lengths = [len(k) for k in r["kept"][0]]
    assert pool.len.tolist() == lengths
    for layer, kept in enumerate(r["kept"]):
        records = pool.caches.pages[layer].reshape(-1, rec)
        for b in range(n):
            # every accepted token's record is what it is at its place in the sequence, whichever way it came there
            pos = torch.arange(lengths[b], dtype=torch.int32, device="cuda")
            got = L.values(records[slots(b, lengths[b])], fmt, 64)
            want, tol = D.appended(kept[b], r["weight"][layer], True, 1e-6, pos, pool.freq, "adjacent", fmt)
            assert ((got - want).abs() <= tol).all()
    for s in r["steps"]:
        before, start = s["before"].tolist(), s["tables"].row_start.tolist()
        for layer, (q, ready, absorbed, out, lse) in enumerate(s["layers"]):
            want, tol = D.norm_rotate(q, r["q_weight"][layer], True, 1e-6, s["pos"], pool.freq, "adjacent")
            assert ((ready.double() - want).abs() <= tol).all()
            records = s["records"][layer].reshape(-1, rec)
            for b, tree in enumerate(s["trees"]):
                values = L.values(records[slots(b, before[b] + len(tree.parents), s["table"].long())], fmt, 64)
                for j, m in enumerate(tree.seen):
                    row = start[b] + j
                    seen = [i for i in range(len(tree.parents)) if m >> i & 1]
                    L.hold(out[row], lse[row], D.attend_row(absorbed[row], values, before[b], seen, example.SCALE, 64))
    # the pages: each in use once or free once
    used = [int(table[b, p]) for b in range(n) for p in range((lengths[b] + 63) // 64)]
    assert sorted(used + pool.free.tolist()) == list(range(pool.caches.pages.shape[1]))


def test_accepted_records_are_those_of_a_plain_append(example):
    """Bit for bit: a draft stored behind the history and moved is the record that appending it alone gives."""
    from sparse_attention_kv_e4m3_gb300 import draft, latent

    r = example.run(record_format="mxfp4", seed=6)
    pool = r["pool"]
    for layer, kept in enumerate(r["kept"]):
        for b, rows in enumerate(kept):
            plain = latent.LatentCache.empty(len(rows) // 64 + 1, 64, "mxfp4")
            at = torch.arange(len(rows), device="cuda")
            draft.csa_latent_append(rows, at, at.int(), plain, pool.freq, weight=r["weight"][layer])
            slots = pool.page_table[b].long()[at // 64] * 64 + at % 64
            assert torch.equal(plain.pages.reshape(-1, 400)[at], pool.caches.pages[layer].reshape(-1, 400)[slots])
