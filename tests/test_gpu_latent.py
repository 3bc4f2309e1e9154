"""The latent-cache operators on the GPU against their 64-bit plain forms (tests/_latent.py,
which derives the tolerances)."""
import math

import pytest
import torch

import _latent as L
from sparse_attention_kv_e4m3_gb300 import latent

pytestmark = pytest.mark.gpu
DEV = "cuda"
PAGE_OOB, RANGE, BAD_REQUEST, LEN_OOB, POOL, ROWS = 1, 4, 16, 32, 64, 128


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_attention_kv_e4m3_gb300 import build

    build.build()
    latent.load()


def ints(v, dtype=torch.int32):
    return torch.tensor(v, dtype=dtype, device=DEV)


def status():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


# ------------------------------------------------------------------ tables

@pytest.mark.parametrize("old,new,extra", [
    ([0], [1], 0), ([64], [0], 2), ([63, 64, 65, 0], [1, 1, 1, 0], 0), ([0, 0, 0], [0, 0, 0], 5),
    ([130, 5, 0, 64, 127], [200, 0, 64, 65, 1], 3), ([0, 7], [4000, 1], 0)])
def test_tables_small(old, new, extra):
    width = max(-(-(a + b) // 64) for a, b in zip(old, new)) + 1
    table, page = [[-1] * width for _ in old], 1000
    for r, a in enumerate(old):
        for p in range(-(-a // 64)):
            table[r][p], page = page, page + 1
    free = list(range(77, 177))
    want_table = [list(r) for r in table]
    want = L.tables(old, new, want_table, free, sum(new) + extra)
    t, st = ints(table), status()
    got = latent.csa_build_tables(ints(old), ints(new), t, ints(free), sum(new) + extra, dev_status=st)
    assert t.tolist() == want_table
    for k, v in want.items():
        assert getattr(got, k).tolist() == v, k
    assert int(st) == 0


@pytest.mark.parametrize("n", [1000, 16384])
def test_tables_many_requests(n):
    g = torch.Generator().manual_seed(n)
    old, new = torch.randint(0, 300, (n,), generator=g).tolist(), torch.randint(0, 9, (n,), generator=g).tolist()
    table, page = [[-1] * 6 for _ in old], 0
    for r, a in enumerate(old):
        for p in range(-(-a // 64)):
            table[r][p], page = page, page + 1
    free = list(range(page, page + 2 * n))
    want_table = [list(r) for r in table]
    want = L.tables(old, new, want_table, free, sum(new) + 1)
    t = ints(table)
    got = latent.csa_build_tables(ints(old), ints(new), t, ints(free), sum(new) + 1)
    assert torch.equal(t.cpu(), torch.tensor(want_table, dtype=torch.int32))
    for k, v in want.items():
        assert getattr(got, k).tolist() == v, k


def test_tables_errors():
    st = status()  # the pool has one page of the three that are needed
    t = ints([[-1, -1], [-1, -1]])
    got = latent.csa_build_tables(ints([0, 0]), ints([65, 1]), t, ints([9]), 66, dev_status=st)
    assert int(st) == POOL and t.tolist() == [[9, -1], [-1, -1]] and got.taken.tolist() == [1]
    assert got.row_slot.tolist() == [9 * 64 + j for j in range(64)] + [-1, -1]
    st = status()  # fewer rows than new records
    got = latent.csa_build_tables(ints([0]), ints([5]), ints([[-1]]), ints([3]), 2, dev_status=st)
    assert int(st) == ROWS and got.row_slot.tolist() == [192, 193] and got.row_start.tolist() == [0, 5]
    st = status()  # lengths below 0 and beyond the table are cut to it
    t = ints([[4, -1], [5, -1]])
    got = latent.csa_build_tables(ints([-3, 100]), ints([2, 1000]), t, ints([7, 8]), 30, dev_status=st)
    assert int(st) == LEN_OOB | PAGE_OOB  # request 1's records 100 .. 127 are on a page that the table does not have
    assert got.row_start.tolist() == [0, 2, 30] and got.kv_start.tolist() == [0, 2, 130]
    assert got.row_slot.tolist() == [7 * 64, 7 * 64 + 1] + [-1] * 28 and t.tolist() == [[7, -1], [5, -1]]
    got = latent.csa_build_tables(ints([]), ints([]), ints([]).reshape(0, 3), ints([]), 2)
    assert got.row_slot.tolist() == [-1, -1] and got.taken.tolist() == [0] and got.row_start.tolist() == [0]


# ------------------------------------------------------------------ writer and reader

def _rows(n, wide, dtype, seed):
    g = gen(seed)
    x = torch.randn(n, wide, generator=g, device=DEV)
    x = x * torch.exp2(torch.randint(-20, 20, (n, 1), generator=g, device=DEV).float())
    x[0] = 0.0
    if n > 3:
        x[1, :32] = 0.0                                             # an empty block beside others
        x[2, :96:3] = -0.0
        x[3, 32:64] = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0] * 4, device=DEV)  # ties
    if n > 6:
        x[4, :512] = torch.randn(512, generator=g, device=DEV) * 2.0 ** -126   # down to subnormals
        x[5] = torch.randn(wide, generator=g, device=DEV) * 2.0 ** -132
        x[6, :512] = torch.randn(512, generator=g, device=DEV).clamp(-3, 3) * 2.0 ** 125
        x[6, 512:] = 1.0
    return x.to(dtype)


@pytest.mark.parametrize("fmt", ["bf16", "mxfp4"])
@pytest.mark.parametrize("rope", [0, 64])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n,pad", [(1, 0), (63, 16), (1000, 256)])
def test_write_and_read(fmt, rope, dtype, n, pad):
    wide, rec = L.LATENT + rope, L.record_bytes(fmt, rope)
    x = _rows(n, wide + 8, dtype, n)[:, :wide]  # rows of a wider tensor
    pages = -(-n // 64) + 2
    buf = torch.full((pages, 64 * rec + pad), 0xA5, dtype=torch.uint8, device=DEV)
    cache = latent.LatentCache(buf, rope, fmt)
    slots = torch.randperm(pages * 64, generator=gen(n + 1), device=DEV)[:n]
    want = buf.clone()
    body = L.make_records(x, fmt, rope)
    for i, s in enumerate(slots.tolist()):
        want[s // 64, s % 64 * rec:(s % 64 + 1) * rec] = body[i]
    st = status()
    latent.csa_latent_write(x, slots, cache, dev_status=st)
    assert int(st) == 0
    assert torch.equal(buf, want)
    # back as histories of two requests whose pages are shuffled
    cut = n // 3
    order = torch.randperm(pages, generator=gen(n + 2), device=DEV).int()
    pt = torch.full((3, pages), -1, dtype=torch.int32, device=DEV)
    pt[0], pt[2] = order, order.flip(0)
    got = latent.csa_latent_read(cache, pt, ints([0, cut, cut, n]), n, dev_status=st)
    rows = buf[:, :64 * rec].reshape(pages, 64, rec)
    back = torch.cat([rows[pt[0].long()].reshape(-1, rec)[:cut], rows[pt[2].long()].reshape(-1, rec)[:n - cut]])
    assert int(st) == 0
    want = L.values(back, fmt, rope).to(torch.bfloat16)
    assert torch.equal(torch.isnan(got), torch.isnan(want)) and torch.equal(got.nan_to_num(), want.nan_to_num())


@pytest.mark.parametrize("fmt", ["bf16", "mxfp4"])
def test_write_refuses_rows(fmt):
    x = torch.ones(7, 576, device=DEV)
    x[1, 3], x[2, 575], x[3, 511] = math.nan, math.inf, -math.inf
    cache = latent.LatentCache.empty(2, 64, fmt)
    cache.pages.zero_()
    st = status()
    latent.csa_latent_write(x, ints([5, 6, 7, 8, -1, 9, 10], torch.int64), cache, dev_status=st)
    assert int(st) == RANGE
    rec = L.record_bytes(fmt, 64)
    full = L.make_records(x[:1], fmt, 64)[0]
    rows = cache.pages.reshape(128, rec)
    for s in range(128):
        assert torch.equal(rows[s], full if s in (5, 9, 10) else torch.zeros_like(full)), s
    st = status()
    latent.csa_latent_write(x[:1].repeat(4, 1), ints([128, -2, 1 << 40, 127], torch.int64), cache, dev_status=st)
    assert int(st) == PAGE_OOB and torch.equal(rows[127], full)


def test_read_errors():
    cache = latent.LatentCache.empty(2, 0, "bf16")
    cache.pages.view(torch.bfloat16).fill_(3.0)
    st = status()
    out = torch.full((140, 512), 9.0, dtype=torch.bfloat16, device=DEV)
    latent.csa_latent_read(cache, ints([[0], [5]]), ints([2, 70, 100]), 140, out=out, dev_status=st)
    # rows 0, 1: before the first request; 66, 67 of request 0 beyond its table; request 1 on a page out of range
    assert int(st) == LEN_OOB | PAGE_OOB
    want = torch.full_like(out, 9.0)
    want[2:66], want[66:100] = 3.0, 0.0
    assert torch.equal(out, want)
    st = status()
    latent.csa_latent_read(cache, ints([[0], [1]]), ints([40, 0, 8]), 3, dev_status=st)
    assert int(st) == LEN_OOB


# ------------------------------------------------------------------ absorbed attention

class Attend:
    """One call's tensors: caches full of records, NaN in every record that no row may see."""

    def __init__(self, lens, heads, rope=64, fmt="bf16", top=0, req=None, pad=0, seed=0, size=1.0, q_pad=0, pt_extra=1):
        g = gen(seed)
        self.rope, self.fmt, self.heads = rope, fmt, heads
        rec, wide = L.record_bytes(fmt, rope), L.LATENT + rope
        nreq = (max(req) + 1) if req else len(lens)
        longest = [max([n for n, r in zip(lens, req or range(len(lens))) if r == k], default=0) for k in range(nreq)]
        counts = [-(-n // 64) for n in longest]
        width = max(counts) + pt_extra
        total = sum(counts) + 2
        order = torch.randperm(total, generator=g, device=DEV).int()
        self.table = torch.full((nreq, width), -7, dtype=torch.int32, device=DEV)
        x = torch.randn(total * 64, wide, generator=g, device=DEV) * size
        body = L.make_records(x, fmt, rope).reshape(total, 64, rec)
        dead = torch.ones(total, 64, dtype=torch.bool, device=DEV)
        at = 0
        for r in range(nreq):
            self.table[r, :counts[r]] = order[at:at + counts[r]]
            for p in range(counts[r]):
                dead[order[at + p], :min(64, longest[r] - 64 * p)] = False
            at += counts[r]
        poison = torch.full((rec,), 0xFF, dtype=torch.uint8, device=DEV)  # NaN in bf16, NaN scales in MXFP4
        body[dead] = poison
        buf = torch.full((total, 64 * rec + pad), 0xFF, dtype=torch.uint8, device=DEV)
        buf[:, :64 * rec] = body.reshape(total, -1)
        self.cache = latent.LatentCache(buf, rope, fmt)
        self.values = L.values(body.reshape(-1, rec), fmt, rope)
        q = torch.randn(len(lens), heads + (1 if q_pad else 0), wide + q_pad, generator=g, device=DEV).to(torch.bfloat16)
        self.q = q[:, :heads, :wide]
        self.lens, self.req = ints(lens), None if req is None else ints(req)
        self.rows = list(zip(lens, req or range(len(lens))))
        self.idx = None
        if top:
            idx = torch.full((len(lens), top), -1, dtype=torch.int32, device=DEV)
            for b, n in enumerate(lens):
                m = min(n, top)
                idx[b, :m] = torch.randperm(n, generator=g, device=DEV)[:m].int() if n else 0
            self.idx = idx
        self.scale = 192 ** -0.5

    def run(self, **kw):
        self.st = status()
        return latent.csa_latent_attend(self.q, self.cache, self.table, self.lens, scale=self.scale, idx=self.idx, row_req=self.req,
                                        dev_status=self.st, **kw)

    def want(self, b):
        n, r = self.rows[b]
        pos = torch.arange(n, device=DEV) if self.idx is None else self.idx[b].long()
        pos = pos[(pos >= 0) & (pos < n)]
        k = self.values[self.table[r].long()[pos // 64] * 64 + pos % 64]
        return L.softmax_out(self.q[b].double(), k, k[:, :L.LATENT], self.scale, k.shape[1])

    def check(self, flags=0, **kw):
        out, lse = self.run(**kw)
        assert int(self.st) == flags
        for b in range(len(self.rows)):
            L.hold(out[b], lse[b], self.want(b))
        return out, lse


@pytest.mark.parametrize("fmt", ["bf16", "mxfp4"])
@pytest.mark.parametrize("rope", [0, 64])
@pytest.mark.parametrize("heads", [1, 5, 16, 64, 65, 128])
def test_attend_whole_history(fmt, rope, heads):
    Attend([0, 1, 63, 64, 65, 127, 300, 1000], heads, rope, fmt, seed=heads).check()


@pytest.mark.parametrize("fmt", ["bf16", "mxfp4"])
@pytest.mark.parametrize("rope", [0, 64])
@pytest.mark.parametrize("heads,top", [(8, 1), (64, 512), (128, 77), (33, 1000)])
def test_attend_positions(fmt, rope, heads, top):
    Attend([2000, 0, 1, 70, 513, 512, 64], heads, rope, fmt, top=top, seed=top).check()


@pytest.mark.parametrize("fmt", ["bf16", "mxfp4"])
def test_attend_positions_with_holes_repeats_and_errors(fmt):
    a = Attend([700, 700, 700, 90], 64, 64, fmt, top=200, seed=5)
    a.idx[0, ::3] = -1                 # holes anywhere
    a.idx[1, 50:100] = a.idx[1, 0]     # a record listed 51 times counts 51 times
    a.idx[2] = -1                      # a mask that leaves the row empty
    a.check()
    a.idx[0, 7], a.idx[1, 9], a.idx[3, 2] = 700, -2, 1 << 30  # left out and reported
    a.check(flags=LEN_OOB)


def test_attend_bad_rows_and_pages():
    for fmt in ("bf16", "mxfp4"):
        a = Attend([300, 300, 300, 300, 300], 16, 64, fmt, req=[0, 1, 2, 1, 0], seed=6)
        out, lse = a.check()
        a.req[2], a.lens[3], a.lens[4] = 3, -5, 64 * a.table.shape[1] + 1
        a.rows[2], a.rows[3] = (0, 0), (0, 0)
        a.lens[4] = 300
        a.check(flags=BAD_REQUEST | LEN_OOB)
        b = Attend([300, 300, 200], 64, 64, fmt, seed=7, pt_extra=0)
        b.lens[0] = 10 ** 6  # cut to the table: 320 records, the last 20 of them NaN
        b.table[0, 4], b.table[1, 1], b.table[2, 0] = 1 << 20, -1, b.cache.pages.shape[0]
        b.rows[0] = (256, 0)
        out, lse = b.run()
        assert int(b.st) == PAGE_OOB | LEN_OOB
        L.hold(out[0], lse[0], b.want(0))
        for r, skip in ((1, 1), (2, 0)):  # the bad page's records are left out
            n = b.rows[r][0]
            pos = torch.tensor([p for p in range(n) if p // 64 != skip], device=DEV)
            k = b.values[b.table[r].long()[pos // 64] * 64 + pos % 64]
            L.hold(out[r], lse[r], L.softmax_out(b.q[r].double(), k, k[:, :512], b.scale, 576))


@pytest.mark.parametrize("fmt", ["bf16", "mxfp4"])
@pytest.mark.parametrize("heads", [16, 128])
def test_attend_long_rows_and_few_rows(fmt, heads):
    Attend([20011], heads, 64, fmt, seed=1).check()
    Attend([9000, 1, 30000], heads, 0, fmt, seed=2).check()


def test_attend_many_rows_of_one_request():
    lens = [(37 * b) % 1500 for b in range(400)]
    Attend(lens, 32, 64, "bf16", req=[0] * 400, seed=3).check()
    Attend(lens, 64, 64, "bf16", top=128, req=[0] * 400, seed=4).check()


@pytest.mark.parametrize("fmt", ["bf16", "mxfp4"])
@pytest.mark.parametrize("order", ["up", "down"])
def test_attend_scores_that_climb(fmt, order):
    """Scores of +-hundreds in ascending and descending order: the running maximum moves all the way."""
    a = Attend([1500, 700], 64, 64, fmt, seed=8, size=4.0)
    for r in range(2):
        n = a.rows[r][0]
        pos = torch.arange(n, device=DEV)
        at = a.table[r].long()[pos // 64] * 64 + pos % 64
        rec = a.cache.pages[:, :64 * a.cache.record_bytes].reshape(-1, a.cache.record_bytes)
        s = (a.values[at] @ a.q[r, 0].double())
        by = s.argsort(descending=order == "down")
        rec[at], a.values[at] = rec[at][by], a.values[at][by]
        a.cache.pages[:, :64 * a.cache.record_bytes] = rec.reshape(a.cache.pages.shape[0], -1)
    a.scale = 1.5
    a.check()


def test_attend_strides_and_padding():
    a = Attend([500, 129], 20, 64, "bf16", pad=16, q_pad=8, seed=9)
    assert not a.q.is_contiguous()
    a.check()
    Attend([500, 129], 20, 64, "mxfp4", pad=48, q_pad=8, top=99, seed=9).check()
    Attend([500, 129], 20, 0, "bf16", pad=1024, top=99, seed=9).check()


def test_attend_offsets_past_32_bits():
    for fmt in ("bf16", "mxfp4"):
        rec = L.record_bytes(fmt, 64)
        pages = (5 << 30) // (64 * rec)
        cache = latent.LatentCache(torch.zeros(pages, 64 * rec, dtype=torch.uint8, device=DEV), 64, fmt)
        x = torch.randn(200, 576, generator=gen(3), device=DEV)
        table = ints([[pages - 1, pages - 3, pages // 2, pages - 2]])
        at = torch.arange(200, device=DEV)
        latent.csa_latent_write(x, table[0].long()[at // 64] * 64 + at % 64, cache)
        k = L.values(L.make_records(x, fmt, 64), fmt, 64)
        assert torch.equal(latent.csa_latent_read(cache, table, ints([0, 200]), 200).double(), k.to(torch.bfloat16).double())
        q = torch.randn(1, 64, 576, generator=gen(4), device=DEV).to(torch.bfloat16)
        want = L.softmax_out(q[0].double(), k, k[:, :512], 0.07, 576)
        for idx in (None, at.int()[None, :]):
            out, lse = latent.csa_latent_attend(q, cache, table, ints([200]), scale=0.07, idx=idx)
            L.hold(out[0], lse[0], want)


def test_attend_same_bits_each_time_on_streams_and_in_graphs():
    for a in (Attend([5000, 300, 0, 77], 64, seed=11), Attend([5000, 300, 0, 77], 128, 64, "mxfp4", seed=11),
              Attend([5000, 300, 0, 77], 64, top=300, seed=11)):
        out, lse = a.check()
        for _ in range(5):
            o, l = a.run()
            assert torch.equal(o, out) and torch.equal(l, lse)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        o, l = torch.zeros_like(out), torch.zeros_like(lse)
        ws = torch.empty(1 << 28, dtype=torch.uint8, device=DEV)
        torch.cuda.synchronize()
        a.run(out=o, lse=l, ws=ws, stream=side)
        side.synchronize()
        assert torch.equal(o, out) and torch.equal(l, lse)
        o.zero_()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            latent.csa_latent_attend(a.q, a.cache, a.table, a.lens, scale=a.scale, idx=a.idx, out=o, lse=l, ws=ws)
        for _ in range(2):
            o.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(o, out) and torch.equal(l, lse)


def test_attend_on_two_streams_at_once():
    """Calls that overlap on two streams, each with the workspace kept for its stream."""
    a, b = Attend([30000, 500], 64, seed=13), Attend([20000, 9000, 3], 128, 64, "mxfp4", seed=14)
    want = [x.check() for x in (a, b)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    torch.cuda.synchronize()
    for _ in range(10):
        for x, s in zip((a, b), streams):
            with torch.cuda.stream(s):
                got.append(latent.csa_latent_attend(x.q, x.cache, x.table, x.lens, scale=x.scale))
    torch.cuda.synchronize()
    for k, (o, l) in enumerate(got):
        assert torch.equal(o, want[k % 2][0]) and torch.equal(l, want[k % 2][1])


def test_attend_more_rows_than_a_block_has_threads():
    """The plan's running sums over rows: several rows a thread, empty rows between others."""
    lens = [(b * 37) % 130 if b % 3 else 0 for b in range(1500)]
    a = Attend(lens, 4, 0, "bf16", req=[b % 5 for b in range(1500)], seed=15)
    out, lse = a.run()
    assert int(a.st) == 0
    for b in list(range(0, 1500, 61)) + [1498, 1499]:
        L.hold(out[b], lse[b], a.want(b))
    assert torch.equal(torch.isneginf(lse[:, 0]).cpu(), torch.tensor(lens) == 0)


# ------------------------------------------------------------------ expanded attention

class Prefill:
    def __init__(self, lq, lk, heads, seed=0, causal=True, size=1.0, contiguous=False):
        g = gen(seed)
        tq, tk = sum(lq), sum(lk)

        def rand(*shape):
            return (torch.randn(*shape, generator=g, device=DEV) * size).to(torch.bfloat16)

        kv, latents = rand(tk, heads, 256), rand(tk, 576)
        self.q, self.kn, self.v, self.kr = rand(tq, heads, 192), kv[..., :128], kv[..., 128:], latents[:, 512:]
        if contiguous:
            self.kn, self.v, self.kr = self.kn.contiguous(), self.v.contiguous(), self.kr.contiguous()
        self.qs, self.ks = [sum(lq[:i]) for i in range(len(lq) + 1)], [sum(lk[:i]) for i in range(len(lk) + 1)]
        self.causal, self.scale, self.heads = causal, 192 ** -0.5, heads

    def run(self, **kw):
        self.st = status()
        return latent.csa_latent_prefill(self.q, self.kn, self.kr, self.v, ints(self.qs), ints(self.ks), scale=self.scale,
                                         causal=self.causal, dev_status=self.st, **kw)

    def check(self, skip=(), rows=None, flags=0):
        out, lse = self.run()
        assert int(self.st) == flags
        for r in range(len(self.qs) - 1):
            if r in skip:
                continue
            (q0, q1), (k0, k1) = self.qs[r:r + 2], self.ks[r:r + 2]
            past = (k1 - k0) - (q1 - q0)
            for h in range(self.heads):
                k = torch.cat([self.kn[k0:k1, h], self.kr[k0:k1]], 1).double()
                q, v = self.q[q0:q1, h].double(), self.v[k0:k1, h].double()
                s = q @ k.t() * self.scale
                live = torch.ones_like(s, dtype=torch.bool)
                if self.causal:
                    live = torch.ones_like(live).tril(past)
                self.hold(out[q0:q1, h], lse[q0:q1, h], s.masked_fill(~live, -math.inf), (q.abs() @ k.abs().t() * self.scale) * live, v)
        return out, lse

    @staticmethod
    def hold(out, lse, s, size, v):
        top = s.amax(1, keepdim=True) if s.shape[1] else torch.full((s.shape[0], 1), -math.inf, dtype=torch.float64, device=DEV)
        empty = torch.isinf(top)
        p = torch.exp(s - torch.where(empty, torch.zeros_like(top), top))
        total = p.sum(1, keepdim=True)
        p = p / total.clamp(min=1e-300)
        want, want_lse = p @ v, (torch.log(total) + top)[:, 0]
        e = (196 * L.F32_HALF * size).amax(1) if s.shape[1] else torch.zeros(s.shape[0], dtype=torch.float64, device=DEV)
        live_s = torch.where(torch.isinf(s), torch.zeros_like(s), s)
        e = e + 16 * L.F32_HALF * (1 + (live_s.abs().amax(1) if s.shape[1] else 0))
        weight = p @ v.abs()
        tol = L.BF16_HALF * want.abs() + (L.BF16_HALF * 1.01 + 2 * e[:, None] + (s.shape[1] + 8) * L.F32_HALF) * weight + 1e-37
        d = (out.double() - want).abs()
        assert (d <= tol).all(), f"out: off by {d.max():.3g}, {float((d / tol).max()):.3g} of the tolerance"
        empty = empty[:, 0]
        assert torch.equal(torch.isneginf(lse), empty)
        dl = torch.where(empty, torch.zeros_like(want_lse), (lse.double() - want_lse).abs())
        assert (dl <= e + 16 * L.F32_HALF * (1 + torch.where(empty, torch.zeros_like(want_lse), want_lse).abs())).all(), f"lse: off by {dl.max():.3g}"


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lq,lk,heads", [
    ([1], [1], 1), ([1, 2, 3], [1, 2, 3], 3), ([128], [128], 2), ([129, 0, 1], [129, 5, 300], 2), ([256, 255, 257], [256, 255, 257], 1),
    ([70, 33], [700, 1000], 4), ([600], [1111], 3), ([5, 300, 64], [5, 2, 0], 2)])
def test_prefill(lq, lk, heads, causal):
    Prefill(lq, lk, heads, seed=len(lq), causal=causal).check()


def test_prefill_contiguous_and_large_scores():
    Prefill([333, 100], [333, 400], 2, seed=5, contiguous=True).check()
    p = Prefill([300], [500], 2, seed=6, size=3.0)
    p.scale = 1.0
    p.check()


def test_prefill_hidden_keys_do_not_matter():
    """NaN and infinities in the keys and values that no row of the other requests sees."""
    p = Prefill([100, 60, 130], [100, 90, 130], 2, seed=7)
    for t in (p.kn, p.v, p.kr):
        t[100:190] = math.nan
        t[110] = math.inf
    p.check(skip=(1,))


def test_prefill_without_keys():
    p = Prefill([5, 200], [0, 0], 2, seed=12)
    out, lse = p.run()
    assert int(p.st) == 0 and not out.any() and torch.isneginf(lse).all()


def test_prefill_many_requests():
    lq = [(13 * i) % 40 for i in range(300)]
    Prefill(lq, [n + (7 * i) % 30 for i, n in enumerate(lq)], 2, seed=8).check()


@pytest.mark.parametrize("causal", [True, False])
def test_prefill_more_items_than_sms(causal):
    """Blocks take over others' items: of all lengths, with one query tile or two, and with tiles that see no key."""
    Prefill([300, 1, 0, 520, 129, 64, 700, 257, 40, 256, 300], [300, 900, 7, 520, 100, 0, 900, 257, 3, 200, 150], 24, seed=13, causal=causal).check()


def test_prefill_more_requests_than_threads():
    lq = [(13 * i) % 40 for i in range(1000)]
    Prefill(lq, [n + (7 * i) % 30 for i, n in enumerate(lq)], 1, seed=14).check()


def test_prefill_output_on_16_bytes():
    p = Prefill([200, 31], [250, 31], 3, seed=15)
    want, want_lse = p.check()
    room = torch.full((231 * 3 * 128 + 16,), 7.0, dtype=torch.bfloat16, device=DEV)
    out, lse = p.run(out=room[8:-8].view(231, 3, 128))
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    assert (room[:8] == 7.0).all() and (room[-8:] == 7.0).all()


def test_prefill_bad_bounds():
    p = Prefill([20, 20, 20], [20, 20, 20], 2, seed=9)
    out = torch.full((60, 2, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    p.ks[3] = 61  # beyond the keys: the last request is left as it is
    p.run(out=out)
    assert int(p.st) == LEN_OOB and (out[40:] == 7.0).all()
    p.check(skip=(2,), flags=LEN_OOB)


def test_prefill_same_bits_each_time_on_streams_and_in_graphs():
    p = Prefill([300, 70], [900, 70], 3, seed=10)
    out, lse = p.check()
    o, l, qs, ks = torch.zeros_like(out), torch.zeros_like(lse), ints(p.qs), ints(p.ks)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    latent.csa_latent_prefill(p.q, p.kn, p.kr, p.v, qs, ks, scale=p.scale, out=o, lse=l, stream=side)
    side.synchronize()
    assert torch.equal(o, out) and torch.equal(l, lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        latent.csa_latent_prefill(p.q, p.kn, p.kr, p.v, qs, ks, scale=p.scale, out=o, lse=l)
    for _ in range(2):
        o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, out) and torch.equal(l, lse)
