"""The indexer's binding with stream=, without a GPU: what a call allocates, fills or copies itself belongs to the
stream that it runs on. Tensors are on the host here and the library only records its calls."""
import contextlib

import pytest
import torch

from sparse_attention_kv_e4m3_gb300 import build, native


class Stream:
    def __init__(self, address):
        self.cuda_stream = address


HOME, SIDE = Stream(0x77), Stream(0x99)


@pytest.fixture
def made(monkeypatch):
    """(storage address, stream entered) of each tensor that a call makes."""
    build.build()
    lib, now, made = native.load(), [None], []

    class Recorder:
        def __getattr__(self, name):
            return getattr(lib, name) if name.endswith("_bytes") else lambda *a: 0

    @contextlib.contextmanager
    def enter(stream):
        before, now[0] = now[0], stream or now[0]
        yield
        now[0] = before

    def note(make):
        def run(*a, **k):
            t = make(*a, **k)
            made.append((t.untyped_storage().data_ptr(), now[0]))
            return t

        return run

    monkeypatch.setattr(native, "load", lambda: Recorder())
    monkeypatch.setattr(torch.cuda, "stream", enter)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: now[0] or HOME)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: None, raising=False)
    for name in ("empty", "full", "zeros"):
        monkeypatch.setattr(torch, name, note(getattr(torch, name)))
    monkeypatch.setattr(torch.Tensor, "contiguous", note(torch.Tensor.contiguous))
    return made


def problem(n=2):
    return native.Problem(q=torch.ones(n, 64, 128, dtype=torch.bfloat16), fused_w=torch.ones(n, 64), kv=torch.ones(4, 64 * 132).byte(),
                          page_table=torch.ones(n, 3).int(), q_len=torch.ones(n).int())


@pytest.mark.parametrize("call", [
    lambda p, **k: native.csa_index_score(p, **k), lambda p, **k: native.csa_index_logits(p, **k),
    lambda p, **k: native.csa_index_score_topk_fused(p, 4, **k), lambda p, **k: native.csa_index_topk(torch.ones(2, 192), p, 4, **k),
    lambda p, **k: native.csa_index_merge_topk(torch.ones(2, 4, 3).int().transpose(1, 2), torch.ones(2, 4, 3).transpose(1, 2), 2, **k),
    lambda p, **k: native.csa_recall_level1([p], **k),
    lambda p, **k: native.csa_index_write_keys(torch.ones(2, 128), torch.ones(2).int(), p.kv, torch.ones(3, 2).int().t(), **k)])
def test_what_a_call_makes_belongs_to_its_stream(made, call):
    call(problem())
    assert made and all(s is None for _, s in made)
    made.clear()
    call(problem(), stream=SIDE)
    assert made and all(s is SIDE for _, s in made)


@pytest.mark.gpu
def test_scores_made_on_a_side_stream_beside_a_busy_current_one(cuda_ok):
    """What the call fills its scores with comes before the scores, whatever the current stream has queued."""
    build.build()
    p = native.Problem(q=torch.ones(2, 64, 128, dtype=torch.bfloat16, device="cuda"), fused_w=torch.ones(2, 64, device="cuda"),
                       kv=torch.zeros(4, 64 * 132, dtype=torch.uint8, device="cuda"),
                       page_table=torch.tensor([[0, 1, 2], [3, 2, 1]], dtype=torch.int32, device="cuda"),
                       q_len=torch.tensor([100, 192], dtype=torch.int32, device="cuda"))
    big, side = torch.ones(256 << 20, device="cuda"), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(4):
        big.mul_(1.0)
    scores = native.csa_index_score(p, stream=side)
    torch.cuda.synchronize()
    assert bool((scores[0, :100] == 0.5).all()) and bool((scores[1] == 0.5).all()) and bool(scores[0, 100:].isnan().all())
