"""The binding of the operators of a step with drafted tokens without a GPU: what it hands to the library, where it takes memory
from, and what it refuses. Tensors are on the host here and the library only records its calls."""
import os
import subprocess
import threading

import pytest
import torch

from sparse_attention_kv_e4m3_gb300 import build, draft, latent
from test_latent_binding import FAKES, Stream, host, ints, made  # noqa: F401


@pytest.fixture
def calls(host, monkeypatch):  # noqa: F811
    """`host` of test_latent_binding, for this module's names too."""
    def want(t, dtype, dims, name, whole=False):
        if t.dtype != dtype or t.dim() != dims or (whole and not t.is_contiguous()):
            raise ValueError(name)
        return t

    host.lib = draft.load()
    monkeypatch.setattr(draft, "_want", want)
    monkeypatch.setattr(draft, "_stream", latent._stream)
    monkeypatch.setattr(draft, "load", lambda: host)
    return host


def cache(layers=0):
    if layers:
        return draft.LayeredCache(torch.zeros(layers, 8, 64 * 1152, dtype=torch.uint8))
    return latent.LatentCache.empty(8, 64, "bf16", device="cpu")


def rotate(n=4, heads=3, dim=128, k_heads=1, **kw):
    q, k = torch.zeros(n, heads, dim, dtype=torch.bfloat16), torch.zeros(n, k_heads, 64, dtype=torch.bfloat16)
    return draft.csa_head_norm_rotate(q, torch.zeros(n, dtype=torch.int32), torch.zeros(32), k=k, **kw)


def append(n=4, **kw):
    return draft.csa_latent_append(torch.zeros(n, 576), torch.zeros(n, dtype=torch.int64), torch.zeros(n, dtype=torch.int32), cache(), torch.zeros(32), **kw)


def attend(rows=3, heads=2, **kw):
    q = torch.zeros(rows, heads, 576, dtype=torch.bfloat16)
    return draft.csa_draft_attend(q, cache(), torch.zeros(2, 4, dtype=torch.int32), ints(5, 6), ints(0, 1, rows), scale=0.1, **kw)


def commit(layers=2, **kw):
    return draft.csa_draft_commit(cache(layers), torch.zeros(2, 4, dtype=torch.int32), ints(5, 6), ints(3, 3), torch.zeros(2, 3, dtype=torch.int32), ints(1, 2), **kw)


@pytest.mark.parametrize("call", [rotate, attend, commit])
def test_outputs_come_from_the_stream_of_the_call(calls, made, call):  # noqa: F811
    side = Stream(0x99)
    made.clear()
    calls.used.clear()
    for t in call(stream=side):
        base = t.untyped_storage().data_ptr()
        assert [s for m, s in made if m.untyped_storage().data_ptr() == base] == [side]
        assert any(s is calls.home for p, s in calls.used if base <= p < base + t.untyped_storage().nbytes())
    assert calls.calls[-1][2][-1] == side.cuda_stream
    calls.used.clear()
    call()
    assert not calls.used and calls.calls[-1][2][-1] == 0


def test_workspaces(calls, made):  # noqa: F811
    """Each call's own, from its stream, also for two calls that are inside the library at once; or the caller's."""
    side = Stream(0x99)
    made.clear()
    attend(stream=side)
    ws, size, on = calls.calls[-1][2]
    assert on == side.cuda_stream and [s for t, s in made if t.data_ptr() == ws] == [side]
    assert size >= draft.draft_attend_workspace_bytes(3, 2, 2, 4)
    mine = torch.zeros(100, dtype=torch.uint8)
    attend(ws=mine)
    assert calls.calls[-1][2][:2] == (mine.data_ptr(), 100)
    both, spans = threading.Barrier(2, timeout=20), []

    def on_call(name, args, rest):
        spans.append((rest[0], rest[0] + rest[1]))
        both.wait()

    calls.on_call = on_call
    threads = [threading.Thread(target=attend, args=(rows,)) for rows in (3, 5)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    (a0, a1), (b0, b1) = spans
    assert a1 <= b0 or b1 <= a0


def test_what_is_handed_over(calls):
    q, k = rotate(eps=0.5, pairing="halves", rope_first=True, rope_scale=2.0, k_norm=False)
    a = calls.calls[-1][1]
    assert (a.q.heads, a.q.dim, a.q.norm, a.k.heads, a.k.dim, a.k.norm) == (3, 128, 1, 1, 64, 0) and a.n == 4
    assert (a.rotation.rope_dim, a.rotation.pairing, a.rotation.scale, a.rope_first, a.eps, a.dtype, a.out_dtype) == (64, 1, 2.0, 1, 0.5, 1, 1)
    assert a.q.out == q.data_ptr() and a.k.out == k.data_ptr() and (a.q.x_row_stride, a.q.x_head_stride) == (384, 128)
    append(norm=False, pairing="halves")
    a = calls.calls[-1][1]
    assert (a.x_stride, a.dtype, a.norm, a.n, a.rotation.rope_dim, a.rotation.pairing, a.weight) == (576, 0, 0, 4, 64, 1, None)
    out, lse = attend()
    a = calls.calls[-1][1]
    assert (a.num_q, a.num_heads, a.num_req, a.pt_stride, a.mask, a.mask_words) == (3, 2, 2, 4, None, 0) and a.out == out.data_ptr() and a.lse == lse.data_ptr()
    wide = torch.zeros(3, 5, dtype=torch.int64)
    attend(mask=wide[:, 1:3])
    a = calls.calls[-1][1]
    assert (a.mask, a.mask_stride, a.mask_words) == (wide.data_ptr() + 8, 5, 2)
    r = commit(3, room=4)
    a = calls.calls[-1][1]
    assert (a.num_layers, a.layer_stride_bytes, a.num_req, a.path_stride, a.room) == (3, 8 * 64 * 1152, 2, 3, 4)
    assert (a.new_len, a.freed, a.n_freed) == tuple(t.data_ptr() for t in r) and [t.shape[0] for t in r] == [2, 4, 1]
    assert commit(1).freed.shape[0] == 8 and calls.calls[-1][1].layer_stride_bytes == 0
    own = draft.Committed(ints(0, 0), ints(0, 0, 0), ints(0))
    assert commit(out=own) is own and calls.calls[-1][1].room == 3


def test_refusals(calls):
    q = torch.zeros(4, 3, 128, dtype=torch.bfloat16)
    pos, freq = torch.zeros(4, dtype=torch.int32), torch.zeros(32)

    def refused(f, kind=ValueError):
        n = len(calls.calls)
        with pytest.raises(kind):
            f()
        assert len(calls.calls) == n

    refused(lambda: draft.csa_head_norm_rotate(q, None, freq))
    refused(lambda: draft.csa_head_norm_rotate(q, pos[:3], freq))
    refused(lambda: draft.csa_head_norm_rotate(q, pos.long(), freq))
    refused(lambda: draft.csa_head_norm_rotate(q, pos, freq.double()))
    refused(lambda: draft.csa_head_norm_rotate(q, pos, freq, pairing="odd"))
    refused(lambda: draft.csa_head_norm_rotate(q.half(), pos, freq), TypeError)
    refused(lambda: draft.csa_head_norm_rotate(q, pos, freq, out_dtype=torch.float16), TypeError)
    refused(lambda: draft.csa_head_norm_rotate(q, pos, freq, k=q[:3]))
    refused(lambda: draft.csa_head_norm_rotate(q, pos, freq, k=q.float()))
    refused(lambda: draft.csa_head_norm_rotate(q, pos, freq, q_weight=torch.zeros(64)))
    refused(lambda: draft.csa_head_norm_rotate(q, pos, freq, q_out=q[:, :2]))
    refused(lambda: draft.csa_head_norm_rotate(q, pos, freq, q_out=q, k=q, k_out=q.float()))
    refused(lambda: draft.csa_head_norm_rotate(q, pos, freq, k_out=q))
    x, slots = torch.zeros(4, 576), torch.zeros(4, dtype=torch.int64)
    refused(lambda: draft.csa_latent_append(x[:, :512], slots, pos, cache(), freq))
    refused(lambda: draft.csa_latent_append(x, slots[:3], pos, cache(), freq))
    refused(lambda: draft.csa_latent_append(x, slots, pos, cache(), freq[:16]))
    refused(lambda: draft.csa_latent_append(x, slots, None, cache(), freq))
    refused(lambda: draft.csa_latent_append(x.half(), slots, pos, cache(), freq), TypeError)
    refused(lambda: draft.csa_latent_append(x, slots, pos, cache(), freq, weight=torch.zeros(576)))
    refused(lambda: attend(mask=torch.zeros(2, 1, dtype=torch.int64)))
    refused(lambda: attend(mask=torch.zeros(3, 0, dtype=torch.int64)))
    refused(lambda: attend(mask=torch.zeros(3, 1, dtype=torch.int32)))
    refused(lambda: attend(ws=torch.zeros(4)))
    refused(lambda: commit(room=-1))
    refused(lambda: commit(out=draft.Committed(ints(0), ints(0), ints(0))))
    refused(lambda: draft.LayeredCache(torch.zeros(0, 8, 64 * 1152, dtype=torch.uint8)))
    refused(lambda: draft.LayeredCache(torch.zeros(2, 8, 64 * 1151, dtype=torch.uint8)))


def test_binding_refuses_host_tensors():
    x = torch.zeros(4, 3, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        draft.csa_head_norm_rotate(x, ints(0, 1, 2, 3), torch.zeros(32))
    with pytest.raises(ValueError):
        draft.LayeredCache(torch.zeros(2, 8, 64 * 1152, dtype=torch.uint8))


RACES = r"""
#include <cstdio>
#include <thread>
#include "csa_draft.h"
static void calls() {
  auto* p = reinterpret_cast<uint8_t*>(0x10000);
  auto* i = reinterpret_cast<int32_t*>(0x10000);
  auto* l = reinterpret_cast<int64_t*>(0x10000);
  auto* f = reinterpret_cast<float*>(0x10000);
  const csa_rotation r = {f, 64, 0, 1.f, 0};
  const csa_heads h = {p, p + 0x10000, f, 1024, 128, 1024, 128, 8, 128, 1, 0};
  for (int format : {CSA_LATENT_BF16, CSA_LATENT_MXFP4}) {
    const csa_latent_cache cache = {p, 8, 64 * 1152, 64, format};
    const csa_append_args w = {cache, p, 576, CSA_KEYS_BF16, 1, 3, l, i, r, f, 1e-6f, 0, nullptr};
    const csa_draft_attend_args a = {cache, p, 16 * 576, 576, 4, 16, i, 4, 4, i, i, nullptr, 0, 0, 0.1f, p, f, nullptr};
    const csa_commit_args c = {cache, 8 * 64 * 1152, 3, 4, i, 4, 5, i, i, i, i, i + 64, i, 7, i, nullptr};
    csa_latent_append(&w, nullptr);
    csa_draft_attend(&a, p, size_t(1) << 40, nullptr);
    csa_draft_commit(&c, nullptr);
  }
  const csa_rotate_args q = {h, h, 3, i, r, CSA_KEYS_BF16, CSA_KEYS_BF16, 0, 1e-6f, nullptr};
  csa_head_norm_rotate(&q, nullptr);
}
int main() {
  std::thread a(calls), b(calls);
  a.join();
  b.join();
  std::printf("done\n");
  return 0;
}
"""


@pytest.mark.skipif(torch.cuda.is_available(), reason="its calls must not reach a GPU: the addresses are made up")
def test_what_the_host_code_keeps_may_be_shared_by_threads(tmp_path):
    """Calls of two threads under the compiler's race detector, without a driver: their launches fail."""
    (tmp_path / "fakes.h").write_text(FAKES)
    (tmp_path / "races.cu").write_text(RACES)
    sources = [str(tmp_path / "races.cu")] + [os.path.join(build.CSRC, f) for f in ("csa_draft_rows.cu", "csa_draft_attend.cu", "csa_latent_cache.cu")]
    exe = str(tmp_path / "races")
    subprocess.run([build.nvcc_path(), "-gencode=arch=compute_103a,code=compute_103a", "-std=c++17", "-t4", "-Xcompiler", "-fsanitize=thread",
                    "-include", str(tmp_path / "fakes.h"), f"-I{build.INCLUDE}", f"-I{build.CSRC}", "-o", exe] + sources, check=True)
    (tmp_path / "known").write_text("race:__device_stub__\n")  # the compiler's launch stubs keep the kernel's address
    ran = subprocess.run([exe], capture_output=True, text=True, env={**os.environ, "TSAN_OPTIONS": f"suppressions={tmp_path}/known"})
    if "FATAL: ThreadSanitizer" in ran.stderr:
        pytest.skip("the race detector does not run here")
    assert "done" in ran.stdout and "csa_draft" not in ran.stderr and "csa_latent" not in ran.stderr, ran.stderr
