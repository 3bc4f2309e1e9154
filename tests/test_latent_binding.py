"""The binding of the latent-cache operators without a GPU: what it hands to the library, where it takes
memory from, and what it refuses. Tensors are on the host here and the library only records its calls;
struct layouts and the library's own refusals are tested in test_latent_abi.py."""
import contextlib
import ctypes
import os
import subprocess
import threading

import pytest
import torch

from sparse_attention_kv_e4m3_gb300 import build, latent

OK = 0


class Recorder:
    """Entry points that note their arguments and launch nothing; sizes come from the library itself."""

    def __init__(self, lib, on_call):
        self.lib, self.on_call, self.calls = lib, on_call, []

    def __getattr__(self, name):
        if name.endswith("_bytes"):
            return getattr(self.lib, name)

        def entry(ref, *rest):
            self.calls.append((name, ref._obj, rest))
            self.on_call(name, ref._obj, rest)
            return OK

        return entry


class Stream:
    def __init__(self, address):
        self.cuda_stream = address


@pytest.fixture
def host(monkeypatch):
    """The binding on host tensors. `host.current()` is the stream that the calling thread has entered, None for its own."""
    build.build()
    state = threading.local()
    host = Recorder(latent.load(), lambda *a: None)
    host.current = lambda: getattr(state, "stream", None)
    host.home = Stream(0x77)

    @contextlib.contextmanager
    def enter(stream):
        before, state.stream = host.current(), stream
        yield
        state.stream = before

    monkeypatch.setattr(latent, "_want", lambda t, *a, **k: t)
    monkeypatch.setattr(latent, "_stream", lambda stream, device: 0 if stream is None else stream.cuda_stream)
    monkeypatch.setattr(latent, "load", lambda: host)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: host.current() or host.home)
    monkeypatch.setattr(torch.cuda, "stream", enter)
    host.used = []  # (address, stream) that a tensor was noted as used on
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: host.used.append((t.data_ptr(), s)), raising=False)
    return host


def ints(*v):
    return torch.tensor(v, dtype=torch.int32)


def attend(rows=3, heads=2, **kw):
    cache = latent.LatentCache.empty(8, 64, "bf16", device="cpu")
    q = torch.zeros(rows, heads, 576, dtype=torch.bfloat16)
    return latent.csa_latent_attend(q, cache, torch.zeros(rows, 4, dtype=torch.int32), torch.ones(rows, dtype=torch.int32), scale=0.1, **kw)


# ------------------------------------------------------------------ workspaces

def test_calls_in_flight_in_two_threads_do_not_share_a_workspace(host):
    """A call is two launches, and the library runs without the interpreter's lock: another thread's call on the
    same stream may be enqueued between them."""
    both = threading.Barrier(2, timeout=20)
    spans = []

    def on_call(name, args, rest):
        ws, size, _ = rest
        spans.append((ws, ws + size))
        both.wait()  # the two calls are inside the library at once

    attend(5)  # whatever a first call may leave behind is there
    host.on_call = on_call
    threads = [threading.Thread(target=attend, args=(rows,)) for rows in (3, 5)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    (a0, a1), (b0, b1) = spans
    assert a1 <= b0 or b1 <= a0


# ------------------------------------------------------------------ streams

@pytest.fixture
def made(host, monkeypatch):
    """(tensor, stream that had been entered) of each tensor that the binding makes with torch.empty."""
    made, empty = [], torch.empty

    def note(*a, **k):
        t = empty(*a, **k)
        made.append((t, host.current()))
        return t

    monkeypatch.setattr(torch, "empty", note)
    return made


def test_workspace_comes_from_the_stream_of_the_call(host, made, monkeypatch):
    """Also while the current stream is captured: the call's stream may be a branch of that capture, and memory given
    back to the capturing stream's order would be handed out again while the branch still uses it."""
    for capturing in (False, True):
        monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: capturing)
        side = Stream(0x99)
        made.clear()
        attend(stream=side)
        ws, _, on = host.calls[-1][2]
        assert on == side.cuda_stream
        assert [s for t, s in made if t.data_ptr() == ws] == [side], capturing


def prefill(tq=4, tk=6, heads=2, **kw):
    def rows(*shape):
        return torch.zeros(*shape, dtype=torch.bfloat16)

    return latent.csa_latent_prefill(rows(tq, heads, 192), rows(tk, heads, 128), rows(tk, 64), rows(tk, heads, 128), ints(0, tq), ints(0, tk),
                                     scale=0.1, **kw)


def tables(n_rows=5, **kw):
    return latent.csa_build_tables(ints(3, 64), ints(4, 1), torch.zeros(2, 3, dtype=torch.int32), ints(7, 8, 9), n_rows, **kw)


def read(n_rows=5, **kw):
    cache = latent.LatentCache.empty(8, 64, "bf16", device="cpu")
    return latent.csa_latent_read(cache, torch.zeros(1, 2, dtype=torch.int32), ints(0, 5), n_rows, **kw)


@pytest.mark.parametrize("call", [attend, prefill, tables, read])
def test_outputs_come_from_the_stream_of_the_call(host, made, call):
    """Memory of the current stream's order may still be read by work queued there. The results are noted as used on
    the current stream too, where the caller waits for them."""
    side = Stream(0x99)
    made.clear()
    host.used.clear()
    got = call(stream=side)
    got = got if isinstance(got, tuple) else (got,)
    for t in got:
        base = t.untyped_storage().data_ptr()
        assert [s for m, s in made if m.untyped_storage().data_ptr() == base] == [side]
        assert any(s is host.home for p, s in host.used if base <= p < base + t.untyped_storage().nbytes())
    host.used.clear()
    call()  # on the current stream: nothing to note
    assert not host.used


# ------------------------------------------------------------------ sizes of zero

@pytest.mark.parametrize("n_rows", [0, 1])
def test_tables_without_rows(host, n_rows):
    """A step that only takes pages, or a captured one of no rows: every table that is not empty has its address."""
    got = tables(n_rows)
    name, args, _ = host.calls[-1]
    assert name == "csa_build_tables" and args.n_rows == n_rows
    for field in ("row_start", "kv_start", "taken") + (("row_req", "row_pos", "row_len", "row_slot") if n_rows else ()):
        assert getattr(args, field) == getattr(got, field).data_ptr() != 0, field


def test_positions_that_list_nothing_are_not_the_whole_history(host):
    """An empty tensor's address is null, which the library reads as "no list"."""
    for stream in (None, Stream(0x99)):
        attend(3, idx=torch.zeros(3, 0, dtype=torch.int32), stream=stream)
        args = host.calls[-1][1]
        assert args.idx and args.top >= 1 and args.idx_stride >= args.top


# ------------------------------------------------------------------ devices

def test_a_call_goes_to_the_current_device_only(monkeypatch):
    """The library launches on the current device: tensors and streams of another one are refused."""
    here, there = torch.device("cuda", 0), torch.device("cuda", 1)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 0x55 + index, raising=False)
    side, far = Stream(0x99), Stream(0x99)
    side.device, far.device = here, there
    assert latent._stream(None, here) == 0x55 and latent._stream(side, here) == 0x99
    for stream, device in ((None, there), (side, there), (far, there), (far, here)):
        with pytest.raises(ValueError):
            latent._stream(stream, device)


# ------------------------------------------------------------------ the library's host code

HARNESS = r"""
#include <cstdio>
#include <cuda_runtime.h>
static int limit = 49152;  // shared memory that the kernel may be launched with, as the driver keeps it for all threads
static cudaError_t set_limit(int bytes) { limit = bytes; return cudaSuccess; }
static cudaError_t number(int* out, int v) { *out = v; return cudaSuccess; }
#define cudaGetDevice(p) number(p, 0)
#define cudaDeviceGetAttribute(p, what, dev) number(p, 152)
#define cudaFuncSetAttribute(kernel, what, bytes) set_limit(static_cast<int>(bytes))
#define cudaOccupancyMaxActiveBlocksPerMultiprocessor(...) cudaErrorUnknown  // ends the call before its launch
#include "csa_latent_cache.cu"
int main() {
  const int requests[] = {16384, 5000, 16384, 100, 4200};
  int32_t* at = reinterpret_cast<int32_t*>(0x1000);
  for (int n : requests) {
    csa_tables_args a = {at, at, n, 8, at, at, 5, 7, at, at, at, reinterpret_cast<int64_t*>(at), at, at, at, nullptr};
    const int status = csa_build_tables(&a, nullptr);
    std::printf("%d %d %d\n", n, status, limit);
  }
  return 0;
}
"""


def test_tables_never_lower_the_kernels_shared_memory_limit(tmp_path):
    """The limit belongs to the kernel, not to the call: another thread's call may be between setting it and its launch."""
    src, exe = tmp_path / "limit.cu", tmp_path / "limit"
    src.write_text(HARNESS)
    subprocess.run([build.nvcc_path(), build.ARCH, "-std=c++17", f"-I{build.INCLUDE}", f"-I{build.CSRC}", "-o", str(exe), str(src)], check=True)
    lines = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split("\n")
    most = 0
    for line in lines[:-1]:
        n, status, limit = map(int, line.split())
        most = max(most, 3 * 4 * (n + 1))
        assert status == 5 and limit >= most, line  # CSA_ERR_CUDA, by the harness


FAKES = r"""
#include <cuda_runtime.h>
static inline cudaError_t number(int* out, int v) { *out = v; return cudaSuccess; }
#define cudaGetDevice(p) number(p, 0)
#define cudaDeviceGetAttribute(p, what, dev) number(p, 152)
#define cudaFuncSetAttribute(...) cudaSuccess
#define cudaOccupancyMaxActiveBlocksPerMultiprocessor(p, ...) number(p, 2)
#define cudaGetLastError() cudaSuccess
"""

RACES = r"""
#include <cstdio>
#include <thread>
#include "csa_latent.h"
static void calls() {
  auto* p = reinterpret_cast<uint8_t*>(0x10000);
  auto* i = reinterpret_cast<int32_t*>(0x10000);
  auto* l = reinterpret_cast<int64_t*>(0x10000);
  auto* f = reinterpret_cast<float*>(0x10000);
  const csa_latent_cache cache = {p, 8, 64 * 1152, 64, CSA_LATENT_BF16};
  const csa_latent_write_args w = {cache, p, 576, CSA_KEYS_BF16, 0, 3, l, nullptr};
  const csa_latent_read_args r = {cache, i, 2, 4, i, 9, p, nullptr};
  const csa_latent_attend_args a = {cache, p, 16 * 576, 576, 4, 16, i, 4, 4, nullptr, i, nullptr, 0, 0, 0.1f, p, f, nullptr};
  const csa_latent_prefill_args e = {p, p, p, p, 768, 192, 1024, 256, 576, 1024, 256, 10, 20, i, i, 2, 4, 1, 0.1f, p, f, nullptr};
  for (int n : {4, 9000}) {
    const csa_tables_args t = {i, i, n, 8, i, i, 5, 7, i, i, i, l, i, i, i, nullptr};
    csa_build_tables(&t, nullptr);
  }
  csa_latent_write(&w, nullptr);
  csa_latent_read(&r, nullptr);
  csa_latent_attend(&a, p, size_t(1) << 40, nullptr);
  csa_latent_prefill(&e, nullptr);
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
    sources = [str(tmp_path / "races.cu")] + [os.path.join(build.CSRC, f"csa_latent_{f}.cu") for f in ("cache", "attend", "prefill")]
    exe = str(tmp_path / "races")
    subprocess.run([build.nvcc_path(), "-gencode=arch=compute_103a,code=compute_103a", "-std=c++17", "-t4", "-Xcompiler", "-fsanitize=thread",
                    "-include", str(tmp_path / "fakes.h"), f"-I{build.INCLUDE}", f"-I{build.CSRC}", "-o", exe] + sources, check=True)
    (tmp_path / "known").write_text("race:__device_stub__\n")  # the compiler's launch stubs keep the kernel's address
    ran = subprocess.run([exe], capture_output=True, text=True, env={**os.environ, "TSAN_OPTIONS": f"suppressions={tmp_path}/known"})
    if "FATAL: ThreadSanitizer" in ran.stderr:
        pytest.skip("the race detector does not run here")
    assert "done" in ran.stdout and "csa_latent" not in ran.stderr, ran.stderr


@pytest.fixture(scope="module")
def lib():
    build.build()
    return latent.load()


@pytest.mark.parametrize("scale", [2.0 ** 127, 3e38])
def test_scales_whose_base_two_form_overflows_are_refused(lib, scale):
    """The kernels compute in powers of two: scale times log2 e has to be finite."""
    at = 0x10000
    cache = latent.CacheArgs(at, 8, 64 * 1152, 64, 0)
    a = latent.AttendArgs(cache, at, 16 * 576, 576, 4, 16, at, 4, 4, None, at, None, 0, 0, scale, at, at, None)
    assert lib.csa_latent_attend(ctypes.byref(a), at, 1 << 40, None) == 1
    p = latent.PrefillArgs(at, at, at, at, 768, 192, 1024, 256, 576, 1024, 256, 10, 20, at, at, 2, 4, 1, scale, at, at, None)
    assert lib.csa_latent_prefill(ctypes.byref(p), None) == 1


@pytest.mark.parametrize("change", [dict(pt_stride=0), dict(pt_stride=-1), dict(top=-1), dict(top=5), dict(idx=16), dict(idx=16, top=-2)])
def test_workspace_of_sizes_that_the_call_refuses_is_0(lib, change):
    sizes = dict(num_q=4, num_heads=16, pt_stride=4)
    assert lib.csa_latent_attend_workspace_bytes(ctypes.byref(latent.AttendArgs(**sizes))) > 0
    assert lib.csa_latent_attend_workspace_bytes(ctypes.byref(latent.AttendArgs(**{**sizes, **change}))) == 0
