"""The draft attention kernel's bounded waits: a wait that runs out ends the call with CSA_DEV_TIMEOUT and leaves the device
clean. As in test_zz_latent_timeout.py no GPU fault, trap or endless loop is involved: the test build of the library limits
the waits to 20 us and holds the loaders back for 200 us, so that the other roles give up; both CTAs of a pair then wait for
the copies that were begun, TMEM is freed, and the call ends. A call of the product library afterwards in the same process must be right."""
import ctypes
import time

import pytest
import torch

from sparse_attention_kv_e4m3_gb300 import draft as D
from test_gpu_draft_attend import Case, draft, latent  # noqa: F401

pytestmark = pytest.mark.gpu
TIMEOUT = 8


@pytest.mark.parametrize("swapped", [False, True])
@pytest.mark.parametrize("fmt", ["bf16", "mxfp4"])
@pytest.mark.parametrize("base,drafts,heads", [([70000, 900, 1], [4, 2, 1], 64), ([700], [5], 16), ([64] * 200, [1] * 200, 128)])
def test_wait_that_runs_out(draft, latent, base, drafts, heads, fmt, swapped):  # noqa: F811
    from sparse_attention_kv_e4m3_gb300 import build

    lib = ctypes.CDLL(build.build_test_variant("timeout"))
    lib.csa_draft_attend.argtypes, lib.csa_draft_attend.restype = D.load().csa_draft_attend.argtypes, ctypes.c_int
    c = Case(latent, base, drafts, heads, fmt=fmt, seed=1)
    if swapped:  # queries that TMA does not reach
        c.q = c.q.transpose(0, 1).contiguous().transpose(0, 1)
    out, lse = c.call(draft)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    o, l = torch.zeros_like(out), torch.zeros_like(lse)
    base_len, start = c.ints(c.base), c.ints(c.start)
    args = D.DraftAttendArgs(c.cache.args, c.q.data_ptr(), c.q.stride(0), c.q.stride(1), c.rows, heads, c.table.data_ptr(), len(base), c.table.shape[1],
                             base_len.data_ptr(), start.data_ptr(), None, 0, 0, c.scale, o.data_ptr(), l.data_ptr(), status.data_ptr())
    ws = torch.empty(1 << 27, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    t = time.monotonic()
    assert lib.csa_draft_attend(ctypes.byref(args), ws.data_ptr(), ws.numel(), torch.cuda.current_stream().cuda_stream) == 0
    torch.cuda.synchronize()
    assert time.monotonic() - t < 3.0 and int(status) & TIMEOUT
    again, lse_again = c.call(draft)
    assert torch.equal(again, out) and torch.equal(lse_again, lse)
