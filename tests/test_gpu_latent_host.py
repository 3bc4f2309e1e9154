"""The latent-cache operators as host programs call them: from several threads, on other streams than the
current one, inside captures that fork. Against the same calls made one after the other on one stream."""
import threading

import pytest
import torch

from sparse_attention_kv_e4m3_gb300 import latent
from test_gpu_latent import DEV, Attend, _lib  # noqa: F401

pytestmark = pytest.mark.gpu


def _in_threads(*work):
    failed = []

    def run(f):
        try:
            f()
        except BaseException as e:  # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=run, args=(f,)) for f in work]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed


def test_attend_in_two_threads_on_one_stream():
    """Calls of two launches each, of different row counts and formats, enqueued on one stream by two threads."""
    cases = [Attend([30000, 500], 64, seed=21), Attend([9000, 3, 20000, 700, 0], 128, 64, "mxfp4", seed=22)]
    want = [c.check() for c in cases]
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    got = [[], []]

    def calls(k):
        c = cases[k]
        with torch.cuda.stream(stream):
            for _ in range(50):
                got[k].append(latent.csa_latent_attend(c.q, c.cache, c.table, c.lens, scale=c.scale))

    _in_threads(lambda: calls(0), lambda: calls(1))
    torch.cuda.synchronize()
    for k in (0, 1):
        assert len(got[k]) == 50
        for out, lse in got[k]:
            assert torch.equal(out, want[k][0]) and torch.equal(lse, want[k][1])
