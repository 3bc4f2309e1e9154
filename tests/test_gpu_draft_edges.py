"""Attention of drafts and the operators around it at the edges: values that are not finite in records that some rows do not
see, tables that change between replays, threads, other streams and branches of captures, calls of other shapes in turn."""
import math
import random

import pytest
import torch

import _draft as D
import _latent as L
from test_gpu_draft_attend import Case, draft, latent, trees  # noqa: F401
from test_gpu_latent_host import _in_threads

pytestmark = pytest.mark.gpu


def status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ not finite

@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("where", ["all", "latent", "rope"])
@pytest.mark.parametrize("base", [0, 60, 130])
def test_bad_draft_beside_rows_that_do_not_see_it(draft, latent, base, where, bad):  # noqa: F811
    """Draft 3's record is not finite. Rows that see it become NaN where its scores do; the others are what they are without it."""
    masks = [0b1, 0b11, 0b111, 0b1000, 0b10111, 0b101000, 0b110111 & ~0b1000, 0]
    c = Case(latent, [base], [8], 12, seed=base + 1)
    clean, clean_lse = c.call(draft, masks)
    c.check(clean, clean_lse, masks)
    pos = base + 3
    page, at = int(c.table[0, pos // 64]), pos % 64
    record = c.cache.pages[page][at * 1152:(at + 1) * 1152].view(torch.bfloat16)
    record[{"all": slice(0, 576), "latent": slice(7, 8), "rope": slice(570, 571)}[where]] = bad
    out, lse = c.call(draft, masks)
    for j, m in enumerate(masks):
        if not m >> 3 & 1:
            assert torch.equal(out[j], clean[j]) and torch.equal(lse[j], clean_lse[j]), j
        elif math.isnan(bad):
            assert out[j].isnan().all() and lse[j].isnan().all()


def test_bad_4_bit_draft_beside_rows_that_do_not_see_it(draft, latent):  # noqa: F811
    masks = [0b1, 0b11, 0b111, 0b1000, 0b10111]
    c = Case(latent, [70], [5], 9, fmt="mxfp4", seed=3)
    clean, clean_lse = c.call(draft, masks)
    page, at = int(c.table[0, 73 // 64]), 73 % 64
    c.cache.pages[page][at * 400 + 256:at * 400 + 272] = 255  # all scales NaN
    out, lse = c.call(draft, masks)
    for j, m in enumerate(masks):
        if m >> 3 & 1:
            assert out[j].isnan().all() and lse[j].isnan().all()
        else:
            assert torch.equal(out[j], clean[j]) and torch.equal(lse[j], clean_lse[j]), j


@pytest.mark.parametrize("block", [0, 7, 8, 15, slice(0, 16)])
@pytest.mark.parametrize("base", [60, 61, 70, 125, 130])
@pytest.mark.parametrize("scale_byte,magnitudes", [(253, (6, 7)), (254, (4, 5, 6, 7)), (254, (0, 4)), (253, (5, 7))])
def test_4_bit_draft_with_infinite_values_beside_rows_that_do_not_see_it(draft, latent, base, block, scale_byte, magnitudes):  # noqa: F811
    """Scale bytes 253 and 254 are powers of two, but 4 x 2^126 and 2 x 2^127 are infinite in bf16. Draft 3 is in the first or the second page of a tile."""
    masks = [0b1, 0b11, 0b111, 0b1000, 0b10111]
    c = Case(latent, [base], [5], 9, fmt="mxfp4", seed=base)
    clean, clean_lse = c.call(draft, masks)
    page, at = int(c.table[0, (base + 3) // 64]), (base + 3) % 64
    record = c.cache.pages[page][at * 400:(at + 1) * 400]
    code = torch.tensor([m | s << 3 for m in magnitudes for s in (0, 1)], dtype=torch.uint8, device="cuda")
    codes = code[torch.arange(32, device="cuda") % len(code)]
    record[:256].view(16, 16)[block] = codes[::2] | codes[1::2] << 4
    record[256:272][block] = scale_byte
    out, lse = c.call(draft, masks)
    for j, m in enumerate(masks):
        if not m >> 3 & 1:
            assert torch.equal(out[j], clean[j]) and torch.equal(lse[j], clean_lse[j]), j


@pytest.mark.parametrize("base", [60, 70])
@pytest.mark.parametrize("scale_byte,magnitude", [(252, 7), (253, 4), (253, 5), (254, 1), (254, 3)])
def test_largest_finite_4_bit_values_of_a_draft(draft, latent, base, scale_byte, magnitude):  # noqa: F811
    """Finite values stay beside infinite ones of their block, for the rows that see them; the queries have nothing there, so that scores stay."""
    masks = [0b1, 0b11, 0b111, 0b1000, 0b11111]
    c = Case(latent, [base], [5], 9, fmt="mxfp4", seed=base)
    c.q[..., 224:256] = 0
    at = int(c.table[0, (base + 3) // 64]) * 64 + (base + 3) % 64
    c.records[at, 112:128], c.records[at, 256 + 7] = 0, scale_byte
    c.records[at, 115] = magnitude | (magnitude | 8) << 4
    c.cache.pages.copy_(c.records.reshape(c.cache.pages.shape))
    out, lse = c.call(draft, masks)
    c.check(out, lse, masks)


@pytest.mark.parametrize("fmt", ["bf16", "mxfp4"])
@pytest.mark.parametrize("base", [0, 61, 70])
def test_draft_whose_score_is_minus_infinity(draft, latent, base, fmt):  # noqa: F811
    """Draft 3 has an infinite value where every query is positive: the rows that see it are what they are without it, or empty where it is all."""
    masks = [0b1, 0b11, 0b111, 0b1000, 0b11111]
    c = Case(latent, [base], [5], 9, fmt=fmt, seed=base)
    c.q[..., 7] = c.q[..., 7].abs() + 0.1
    want, want_lse = c.call(draft, [m & ~0b1000 for m in masks])
    page, at, rec = int(c.table[0, (base + 3) // 64]), (base + 3) % 64, c.cache.record_bytes
    record = c.cache.pages[page][at * rec:(at + 1) * rec]
    if fmt == "bf16":
        record.view(torch.bfloat16)[7] = -math.inf
    else:
        record[:16] = 0
        record[3], record[256] = 15 << 4, 254
    out, lse = c.call(draft, masks)
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    if base == 0:
        assert not out[3].any() and torch.isneginf(lse[3]).all()


def test_queries_that_are_not_finite_stay_in_their_row(draft, latent):  # noqa: F811
    c = Case(latent, [300], [5], 30, seed=4)
    clean, clean_lse = c.call(draft)
    c.q[2, 7, 100] = math.nan
    out, lse = c.call(draft)
    assert out[2, 7].isnan().all() and lse[2, 7].isnan()
    out[2, 7], lse[2, 7] = clean[2, 7], clean_lse[2, 7]
    assert torch.equal(out, clean) and torch.equal(lse, clean_lse)


# ------------------------------------------------------------------ sizes and strides

@pytest.mark.parametrize("fmt", ["bf16", "mxfp4"])
@pytest.mark.parametrize("heads", [5, 64, 100])
def test_queries_in_other_orders(draft, latent, heads, fmt):  # noqa: F811
    """Head-major queries, rows with values behind them, one head of a wider tensor, one row."""
    c = Case(latent, [150, 7], [9, 2], heads, fmt=fmt, seed=5)
    want, want_lse = c.call(draft)
    c.check(want, want_lse, words=None)
    swapped = c.q.transpose(0, 1).contiguous().transpose(0, 1)
    wide = torch.full((11, heads, 600), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[..., 8:584] = c.q
    for q in (swapped, wide[..., 8:584]):
        out, lse = c.call(draft, q=q)
        assert torch.equal(out, want) and torch.equal(lse, want_lse)
    one, one_lse = draft.csa_draft_attend(wide[:, 3:4, 8:584], c.cache, c.table, c.ints(c.base), c.ints(c.start), scale=c.scale)
    assert torch.equal(one, want[:, 3:4]) and torch.equal(one_lse, want_lse[:, 3:4])


@pytest.mark.parametrize("fmt", ["bf16", "mxfp4"])
def test_more_requests_than_threads(draft, latent, fmt):  # noqa: F811
    rng = random.Random(6)
    base, drafts = [rng.randint(0, 90) for _ in range(1300)], [rng.choice([0, 1, 1, 2, 5]) for _ in range(1300)]
    c = Case(latent, base, drafts, 3, fmt=fmt, seed=6)
    out, lse = c.call(draft)
    rows = set(rng.sample(range(1300), 60)) | {0, 1299}
    for r in rows:
        values = c.values(r)
        for j in range(drafts[r]):
            row = c.start[r] + j
            L.hold(out[row], lse[row], D.attend_row(c.q[row], values, base[r], range(j + 1), c.scale, 64))


@pytest.mark.parametrize("fmt", ["bf16", "mxfp4"])
def test_many_units_of_one_request(draft, latent, fmt):  # noqa: F811
    """64 drafts of 128 heads: 64 units, one history."""
    c = Case(latent, [1500], [64], 128, fmt=fmt, seed=7)
    masks = trees(random.Random(8), [64])
    out, lse = c.call(draft, masks)
    c.check(out, lse, masks, rows=[0, 1, 31, 32, 62, 63])


def test_sixteen_words_of_drafts(draft, latent):  # noqa: F811
    n = 1024
    rng = random.Random(9)
    masks = [rng.getrandbits(1024) & ((1 << (j + 1)) - 1) for j in range(n)]
    c = Case(latent, [77], [n], 1, seed=9)
    out, lse = c.call(draft, masks, 16)
    c.check(out, lse, masks, 16, rows=[0, 1, 63, 64, 65, 500, 511, 512, 1022, 1023])


def test_no_lse(draft, latent):  # noqa: F811
    import ctypes

    c = Case(latent, [3000, 40], [3, 2], 8, seed=10)
    want, _ = c.call(draft)
    out, base, start = torch.zeros_like(want), c.ints(c.base), c.ints(c.start)
    a = draft.DraftAttendArgs(c.cache.args, c.q.data_ptr(), 8 * 576, 576, 5, 8, c.table.data_ptr(), 2, c.table.shape[1], base.data_ptr(), start.data_ptr(),
                              None, 0, 0, c.scale, out.data_ptr(), None, None)
    n = draft.load().csa_draft_attend_workspace_bytes(ctypes.byref(a))
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    assert draft.load().csa_draft_attend(ctypes.byref(a), ws.data_ptr(), n, torch.cuda.current_stream().cuda_stream) == 0
    assert torch.equal(out, want)


@pytest.mark.parametrize("fmt", ["bf16", "mxfp4"])
@pytest.mark.parametrize("base,drafts,heads", [([70000, 900, 1], [4, 2, 1], 64), ([200] * 400, [1] * 400, 128), ([300, 40, 700, 129] * 60, [2, 3, 1, 4] * 60, 64),
                                               ([5000] * 40, [3] * 40, 64)])
def test_the_same_bits_again_and_again(draft, latent, base, drafts, heads, fmt):  # noqa: F811
    """Runs of pieces of one to many tiles, in which the loaders go from one piece to the next while the last one is still being read;
    by both ways in which the queries come."""
    c = Case(latent, base, drafts, heads, fmt=fmt, seed=20)
    out, lse = c.call(draft)
    c.check(out, lse, words=None, rows=[0]) if len(base) < 10 else None
    swapped = c.q.transpose(0, 1).contiguous().transpose(0, 1)
    busy = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    for k in range(25):
        if k % 5 == 0:
            busy.fill_(k)  # cold caches: other waits are the long ones
        again, lse_again = c.call(draft, q=swapped if k % 2 else c.q)
        assert torch.equal(again, out) and torch.equal(lse_again, lse), k


@pytest.mark.parametrize("fmt", ["bf16", "mxfp4"])
@pytest.mark.parametrize("base,drafts,heads", [([200] * 400, [1] * 400, 128), ([300, 40, 700, 129] * 60, [2, 3, 1, 4] * 60, 64), ([5000] * 40, [3] * 40, 64)])
def test_runs_of_several_pieces_against_the_64_bit_form(draft, latent, base, drafts, heads, fmt):  # noqa: F811
    """The shapes above whose runs go through several pieces: the first and last requests and a sample, each draft of them, by both ways of the queries."""
    c = Case(latent, base, drafts, heads, fmt=fmt, seed=23)
    rows = sorted(set(random.Random(24).sample(range(len(base)), 20)) | {0, 1, len(base) - 2, len(base) - 1})
    for q in (c.q, c.q.transpose(0, 1).contiguous().transpose(0, 1)):
        out, lse = c.call(draft, q=q)
        for r in rows:
            values = c.values(r)
            for j in range(drafts[r]):
                row = c.start[r] + j
                L.hold(out[row], lse[row], D.attend_row(c.q[row], values, base[r], range(j + 1), c.scale, 64))


def test_a_call_of_more_than_a_second(draft, latent):  # noqa: F811
    """The waits' limit is a second: none may begin with a run and end with it. A history of 500000 records, whose pages are 40 in turn, and
    16384 drafts of 128 heads: 2.3 x 10^15 operations."""
    n, heads, base, distinct = 16384, 128, 500000, 40
    c = Case(latent, [distinct * 64 - 64], [64], 1, seed=21)
    pages = c.table[0, :distinct]
    table = pages.repeat((base + n + 63) // 64 // distinct + 1)[None, :(base + n + 63) // 64].contiguous()
    g = torch.Generator(device="cuda").manual_seed(22)
    q = torch.empty(n, heads, 576, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    bad = torch.zeros(1, dtype=torch.int32, device="cuda")
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    begin.record()
    out, lse = draft.csa_draft_attend(q, c.cache, table, c.ints([base]), c.ints([0, n]), scale=1.0, dev_status=bad)
    end.record()
    torch.cuda.synchronize()
    assert int(bad) == 0 and begin.elapsed_time(end) > 1000
    pos = torch.arange(base + n, device="cuda")
    values = L.values(c.records[table[0].long()[pos // 64] * 64 + pos % 64], "bf16", 64)
    for j in (0, 1, 8191, n - 1):
        k = values[:base + j + 1]
        for h in (0, 127):
            L.hold(out[j, h:h + 1], lse[j, h:h + 1], L.softmax_out(q[j, h:h + 1].double(), k, k[:, :512], 1.0, 576))


# ------------------------------------------------------------------ graphs, streams, threads

@pytest.mark.parametrize("fmt", ["bf16", "mxfp4"])
def test_replays_with_other_lengths_and_masks(draft, latent, fmt):  # noqa: F811
    """A captured call whose tables, lengths and masks are written between the replays, padding rows among them."""
    c = Case(latent, [2000, 500, 90], [6, 4, 0], 16, fmt=fmt, seed=11, spare_rows=4)
    base, start, mask = c.ints(c.base), c.ints(c.start), D.words([0] * 14, 1, "cuda")
    out, lse = torch.zeros(14, 16, 512, dtype=torch.bfloat16, device="cuda"), torch.zeros(14, 16, device="cuda")
    ws = torch.empty(draft.draft_attend_workspace_bytes(14, 16, 3, c.table.shape[1]), dtype=torch.uint8, device="cuda")

    def call():
        draft.csa_draft_attend(c.q, c.cache, c.table, base, start, scale=c.scale, mask=mask, out=out, lse=lse, ws=ws)

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    rng = random.Random(12)
    total = [b + n for b, n in zip(c.base, c.drafts)]
    for _ in range(6):
        c.drafts = [rng.randint(0, 4) for _ in range(3)]
        c.base = [rng.randint(0, t - n) for t, n in zip(total, c.drafts)]
        c.start = [sum(c.drafts[:k]) for k in range(4)]
        masks = trees(rng, c.drafts)
        base.copy_(c.ints(c.base)), start.copy_(c.ints(c.start)), mask.copy_(D.words(masks + [0] * (14 - len(masks)), 1, "cuda"))
        out.fill_(7.0)
        ws.fill_(255)
        graph.replay()
        c.check(out, lse, masks) if masks else None
        assert (out[c.start[-1]:] == 7).all()


def test_two_graphs_with_one_workspace(draft, latent):  # noqa: F811
    """Replayed in turn on one stream, of different shapes: nothing in the workspace outlives a call."""
    a, b = Case(latent, [9000, 30], [5, 2], 16, seed=13), Case(latent, [700, 700, 64], [3, 9, 1], 64, fmt="mxfp4", seed=14)
    want = [a.call(draft), b.call(draft)]
    size = max(draft.draft_attend_workspace_bytes(c.rows, c.heads, len(c.base), c.table.shape[1]) for c in (a, b))
    ws, outs, graphs, keep = torch.empty(size, dtype=torch.uint8, device="cuda"), [], [], []
    for c in (a, b):
        o = torch.empty(c.rows, c.heads, 512, dtype=torch.bfloat16, device="cuda"), torch.empty(c.rows, c.heads, device="cuda")
        args = c.ints(c.base), c.ints(c.start)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            draft.csa_draft_attend(c.q, c.cache, c.table, *args, scale=c.scale, out=o[0], lse=o[1], ws=ws)
        outs.append(o), graphs.append(g), keep.append(args)
    for k in (0, 1, 0, 0, 1, 1, 0):
        outs[k][0].zero_()
        graphs[k].replay()
        assert torch.equal(outs[k][0], want[k][0]) and torch.equal(outs[k][1], want[k][1])


def test_calls_of_two_threads_on_one_stream(draft, latent):  # noqa: F811
    cases = [Case(latent, [30000, 500], [4, 9], 64, seed=15), Case(latent, [9000, 3, 2000], [1, 5, 0], 100, fmt="mxfp4", seed=16)]
    want = [c.call(draft) for c in cases]
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    got = [[], []]

    def calls(k):
        with torch.cuda.stream(stream):
            for _ in range(40):
                got[k].append(cases[k].call(draft))

    _in_threads(lambda: calls(0), lambda: calls(1))
    torch.cuda.synchronize()
    for k in (0, 1):
        assert len(got[k]) == 40
        for out, lse in got[k]:
            assert torch.equal(out, want[k][0]) and torch.equal(lse, want[k][1])


def test_two_calls_at_once(draft, latent):  # noqa: F811
    """On two streams, each with its own workspace."""
    a, b = Case(latent, [20000], [4], 64, seed=17), Case(latent, [15000, 300], [3, 3], 16, fmt="mxfp4", seed=18)
    want = a.call(draft), b.call(draft)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [[], []]
    for _ in range(20):
        for k, c in enumerate((a, b)):
            got[k].append(c.call(draft, stream=streams[k]))
    torch.cuda.synchronize()
    for k in (0, 1):
        for out, lse in got[k]:
            assert torch.equal(out, want[k][0]) and torch.equal(lse, want[k][1])


def test_every_operator_on_a_branch_of_a_capture(draft, latent):  # noqa: F811
    """With the outputs that the calls make themselves."""
    c = Case(latent, [900, 70], [5, 3], 16, seed=19)
    g = torch.Generator(device="cuda").manual_seed(1)
    x, q = torch.randn(8, 576, generator=g, device="cuda"), torch.randn(8, 16, 192, generator=g, device="cuda")
    k, pos, freq = torch.randn(8, 1, 64, generator=g, device="cuda"), torch.arange(8, dtype=torch.int32, device="cuda"), D.freqs(64, device="cuda")
    slots, base, start, drafts = torch.arange(8, device="cuda"), c.ints(c.base), c.ints(c.start), c.ints(c.drafts)
    path, path_len = c.ints([[1, 3], [0, 2]]), c.ints([2, 2])
    pages, moved = c.cache.pages.clone(), c.cache.pages.clone()

    def calls(**kw):
        own, other = latent.LatentCache(pages, 64, "bf16"), latent.LatentCache(moved, 64, "bf16")
        draft.csa_latent_append(x, slots, pos, own, freq, **kw)
        rotated = draft.csa_head_norm_rotate(q, pos, freq, k=k, **kw)
        out = draft.csa_draft_attend(c.q, c.cache, c.table, base, start, scale=c.scale, **kw)
        done = draft.csa_draft_commit(other, c.table, base, drafts, path, path_len, **kw)
        return (*rotated, *out, *done)

    want = [t.clone() for t in calls()]
    want_pages, want_moved = pages.clone(), moved.clone()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        got = calls(stream=side)
        main.wait_stream(side)
    for _ in range(3):
        for t in got:
            t.zero_()
        pages.copy_(c.cache.pages)
        moved.copy_(c.cache.pages)
        graph.replay()
        torch.cuda.synchronize()
        for t, w in zip(got, want):
            assert torch.equal(t, w)
        assert torch.equal(pages, want_pages) and torch.equal(moved, want_moved)
