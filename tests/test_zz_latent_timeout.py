"""The latent attention kernels' bounded waits: a wait that runs out ends the call with
CSA_DEV_TIMEOUT and leaves the device clean.

As in test_zz_timeout.py, no GPU fault, trap or endless loop is involved. The same test build of
the library (pipeline waits limited to 20 us) holds the kernels' loaders back for 200 us, so that the
softmax and the MMA roles give up waiting for the first tile; the loaders then find the abort flag, wait for
the copies they have begun, TMEM is freed, and the call ends. A call of the product library afterwards in
the same process must be right, which it could not be with TMEM left allocated or a copy in flight."""
import ctypes
import time

import pytest
import torch

import _latent as L
from sparse_attention_kv_e4m3_gb300 import latent
from test_gpu_latent import DEV, Attend, Prefill, ints, status

pytestmark = pytest.mark.gpu
TIMEOUT = 8


@pytest.fixture(scope="module")
def timeout_lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_attention_kv_e4m3_gb300 import build

    build.build()
    lib, product = ctypes.CDLL(build.build_test_variant("timeout")), latent.load()
    for name in ("csa_latent_attend", "csa_latent_prefill"):
        getattr(lib, name).argtypes = getattr(product, name).argtypes
        getattr(lib, name).restype = ctypes.c_int
    return lib


def _timed(call):
    torch.cuda.synchronize()
    t = time.monotonic()
    assert call() == 0
    torch.cuda.synchronize()
    return time.monotonic() - t


# whole histories in runs (TMA), short units in clusters, 4-bit records, listed positions
@pytest.mark.parametrize("case", [
    dict(lens=[70000, 900, 1], fmt="bf16"), dict(lens=[700, 64], fmt="bf16"), dict(lens=[40000, 5], fmt="mxfp4"),
    dict(lens=[3000] * 200, fmt="bf16", top=512, req=[0] * 200)])
def test_attend_wait_that_runs_out(timeout_lib, case):
    a = Attend(case["lens"], 64, 64, case["fmt"], top=case.get("top", 0), req=case.get("req"), seed=1)
    out, lse = a.check()  # the product library
    st = status()
    o, l = torch.zeros_like(out), torch.zeros_like(lse)
    ws = torch.empty(1 << 27, dtype=torch.uint8, device=DEV)
    args = latent.AttendArgs(a.cache.args, a.q.data_ptr(), a.q.stride(0), a.q.stride(1), a.q.shape[0], 64, a.table.data_ptr(),
                             a.table.shape[0], a.table.shape[1], None if a.req is None else a.req.data_ptr(), a.lens.data_ptr(),
                             None if a.idx is None else a.idx.data_ptr(), 0 if a.idx is None else a.idx.stride(0), case.get("top", 0),
                             a.scale, o.data_ptr(), l.data_ptr(), st.data_ptr())
    took = _timed(lambda: timeout_lib.csa_latent_attend(ctypes.byref(args), ws.data_ptr(), ws.numel(), torch.cuda.current_stream().cuda_stream))
    assert int(st) & TIMEOUT and took < 1.0
    again, lse_again = a.run()
    assert torch.equal(again, out) and torch.equal(lse_again, lse) and int(a.st) == 0


def test_prefill_wait_that_runs_out(timeout_lib):
    p = Prefill([1000, 300, 5], [3000, 300, 5], 4, seed=2)
    out, lse = p.check()
    st, qs, ks = status(), ints(p.qs), ints(p.ks)
    o, l = torch.zeros_like(out), torch.zeros_like(lse)
    args = latent.PrefillArgs(p.q.data_ptr(), p.kn.data_ptr(), p.kr.data_ptr(), p.v.data_ptr(), p.q.stride(0), p.q.stride(1),
                              p.kn.stride(0), p.kn.stride(1), p.kr.stride(0), p.v.stride(0), p.v.stride(1), p.q.shape[0],
                              p.kn.shape[0], qs.data_ptr(), ks.data_ptr(), 3, 4, 1, p.scale, o.data_ptr(), l.data_ptr(), st.data_ptr())
    took = _timed(lambda: timeout_lib.csa_latent_prefill(ctypes.byref(args), torch.cuda.current_stream().cuda_stream))
    assert int(st) & TIMEOUT and took < 1.0
    again, lse_again = p.run()
    assert torch.equal(again, out) and torch.equal(lse_again, lse) and int(p.st) == 0
