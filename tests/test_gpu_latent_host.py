"""The latent-cache operators as host programs call them: from several threads, on other streams than the
current one, inside captures that fork. Against the same calls made one after the other on one stream."""
import threading

import pytest
import torch

from sparse_attention_kv_e4m3_gb300 import latent
from test_gpu_latent import DEV, Attend, Prefill, _lib, ints  # noqa: F401

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


@pytest.mark.parametrize("fmt", ["bf16", "mxfp4"])
def test_attend_on_a_branch_of_a_capture(fmt):
    """The call goes to a stream forked from the capturing one, which allocates and fills memory meanwhile."""
    a = Attend([30000, 500, 9000], 64, 64, fmt, seed=23)
    want, want_lse = a.check()
    out, lse = torch.zeros_like(want), torch.zeros_like(want_lse)
    size = latent.attend_workspace_bytes(3, 64, a.table.shape[1])
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        latent.csa_latent_attend(a.q, a.cache, a.table, a.lens, scale=a.scale, out=out, lse=lse, stream=side)
        rest = [torch.empty(size, dtype=torch.uint8, device=DEV).fill_(255) for _ in range(8)]
        main.wait_stream(side)
    for _ in range(20):
        out.zero_()
        lse.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, want_lse)
    assert all(bool((r == 255).all()) for r in rest)


def test_results_made_on_another_stream():
    """The current stream's queued work still reads memory that it has given back when a call on a side stream makes
    its outputs."""
    a = Attend([700, 90], 64, 64, "bf16", seed=24)
    want, want_lse = a.check()
    side = torch.cuda.Stream()
    big = torch.randn(64 << 20, device=DEV)
    for _ in range(10):
        torch.cuda.synchronize()
        side.wait_stream(torch.cuda.current_stream())
        old = [torch.full_like(want, 3.0) for _ in range(4)]
        for _ in range(4):
            big.mul_(1.0)  # keeps the current stream busy before it reads `old`
        read = [t.clone() for t in old]
        del old
        out, lse = latent.csa_latent_attend(a.q, a.cache, a.table, a.lens, scale=a.scale, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        copy = out.clone()
        del out
        again = latent.csa_latent_attend(a.q, a.cache, a.table, a.lens, scale=2 * a.scale, stream=side)[0]
        torch.cuda.synchronize()
        assert all(bool((t == 3.0).all()) for t in read)
        assert torch.equal(copy, want) and torch.equal(lse, want_lse) and not torch.equal(again, want)


def test_tables_without_rows():
    for own in (False, True):
        st, t = torch.zeros(1, dtype=torch.int32, device=DEV), torch.full((2, 3), -1, dtype=torch.int32, device=DEV)
        out = latent.empty_tables(2, 0) if own else None
        got = latent.csa_build_tables(ints([0, 0]), ints([65, 0]), t, ints([5, 6, 7]), 0, out=out, dev_status=st)
        assert got.row_start.tolist() == got.kv_start.tolist() == [0, 65, 65] and got.taken.tolist() == [2]
        assert t.tolist() == [[5, 6, -1], [-1, -1, -1]] and got.row_slot.shape == (0,)
        assert int(st) == 128  # records without a row of their own


@pytest.mark.parametrize("fmt", ["bf16", "mxfp4"])
def test_attend_with_no_positions(fmt):
    a = Attend([300, 0, 70], 16, 64, fmt, seed=25)
    a.idx = torch.zeros(3, 0, dtype=torch.int32, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (None, side):
        out, lse = a.run(stream=stream)
        torch.cuda.synchronize()
        assert int(a.st) == 0 and not out.any() and bool(torch.isneginf(lse).all())


def test_tables_of_many_sizes_in_threads():
    """Tables of more requests than the default limit of shared memory holds, of other sizes in each thread."""
    def calls(n):
        zero, one = torch.zeros(n, dtype=torch.int32, device=DEV), torch.ones(n, dtype=torch.int32, device=DEV)
        table, free = torch.full((n, 1), -1, dtype=torch.int32, device=DEV), torch.arange(n, dtype=torch.int32, device=DEV)
        for _ in range(1500):
            got = latent.csa_build_tables(zero, one, table, free, n)
        assert torch.equal(got.row_slot, 64 * torch.arange(n, device=DEV)) and int(got.taken) == n

    _in_threads(*(lambda n=n: calls(n) for n in (16384, 4200, 9000, 16384)))
    torch.cuda.synchronize()


def test_results_made_on_a_branch_of_a_capture():
    """Every operator on a stream forked from the capturing one, with the outputs that the calls make themselves."""
    a, p = Attend([900, 70], 16, 64, "bf16", seed=26), Prefill([40, 9], [60, 9], 2, seed=27)
    qs, ks, start = ints(p.qs), ints(p.ks), ints([0, 900, 970])
    old, new, free = ints([900, 70]), ints([3, 0]), ints([50, 51])

    def calls(**kw):
        table = a.table.clone() if not kw else own_table
        t = latent.csa_build_tables(old, new, table, free, 4, **kw)
        rows = latent.csa_latent_read(a.cache, a.table, start, 970, **kw)
        o = latent.csa_latent_attend(a.q, a.cache, a.table, a.lens, scale=a.scale, **kw)
        none = latent.csa_latent_attend(a.q, a.cache, a.table, a.lens, scale=a.scale, idx=old.reshape(2, 1)[:, :0], **kw)
        e = latent.csa_latent_prefill(p.q, p.kn, p.kr, p.v, qs, ks, scale=p.scale, **kw)
        return (table, *t, rows, *o, *none, *e)

    own_table = a.table.clone()
    want = calls()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        got = calls(stream=side)
        main.wait_stream(side)
    for _ in range(3):
        for g in got[1:]:
            g.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert torch.equal(g, w)
