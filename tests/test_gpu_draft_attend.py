"""Attention of drafted tokens over the paged latent cache on the GPU, against its 64-bit form."""
import random

import pytest
import torch

import _draft as D
import _latent as L

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def draft():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_attention_kv_e4m3_gb300 import build

    build.build()
    from sparse_attention_kv_e4m3_gb300 import draft

    return draft


@pytest.fixture(scope="module")
def latent(draft):
    from sparse_attention_kv_e4m3_gb300 import latent

    return latent


class Case:
    """Histories in shuffled pages full of records, NaN in every page's records that no request has."""

    def __init__(self, latent, base, drafts, heads, rope=64, fmt="bf16", seed=0, spare_rows=0, pad=0, extra_width=1, grow=1.0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.base, self.drafts, self.heads, self.rope, self.fmt = base, drafts, heads, rope, fmt
        need = [(b + n + 63) // 64 for b, n in zip(base, drafts)]
        width, pages = max(need + [0]) + extra_width, sum(need) + 2
        order = torch.randperm(pages, generator=g, device="cuda")
        self.table = torch.full((len(base), width), -1, dtype=torch.int32, device="cuda")
        at = 0
        rec = L.record_bytes(fmt, rope)
        x = torch.randn(pages * 64, 512 + rope, generator=g, device="cuda") * grow
        records = L.make_records(x.to(torch.bfloat16), fmt, rope).reshape(pages, 64, rec)
        live = torch.zeros(pages, 64, dtype=torch.bool, device="cuda")
        for r, n in enumerate(need):
            self.table[r, :n] = order[at:at + n].int()
            total = base[r] + drafts[r]
            for p in range(n):
                live[order[at + p], :max(0, min(64, total - 64 * p))] = True
            at += n
        nan = torch.full((rec,), 0xFF, dtype=torch.uint8, device="cuda")  # NaN as bf16, and as a scale byte
        records = torch.where(live[..., None], records, nan)
        pool = torch.full((pages, 64 * rec + pad), 0xFF, dtype=torch.uint8, device="cuda")
        pool[:, :64 * rec] = records.reshape(pages, -1)
        self.cache = latent.LatentCache(pool, rope, fmt)
        self.start = [sum(drafts[:k]) for k in range(len(drafts) + 1)]
        self.rows = self.start[-1] + spare_rows
        self.q = torch.randn(self.rows, heads, 512 + rope, generator=g, device="cuda").to(torch.bfloat16)
        self.scale = (128 + rope) ** -0.5
        self.records = records.reshape(-1, rec)

    def ints(self, v):
        return torch.tensor(v, dtype=torch.int32, device="cuda")

    def values(self, r):
        total = self.base[r] + self.drafts[r]
        pos = torch.arange(total, device="cuda")
        return L.values(self.records[self.table[r].long()[pos // 64] * 64 + pos % 64], self.fmt, self.rope)

    def call(self, draft, masks=None, words=1, **kw):
        m = None if masks is None else D.words(masks + [0] * (self.rows - len(masks)), words, "cuda")
        args = dict(scale=self.scale, mask=m)
        args.update(kw)
        return draft.csa_draft_attend(args.pop("q", self.q), self.cache, args.pop("page_table", self.table), self.ints(self.base), self.ints(self.start), **args)

    def check(self, out, lse, masks=None, words=1, rows=None):
        masks = masks or [m for n in self.drafts for m in D.chain(n)]
        for r, n in enumerate(self.drafts):
            values = self.values(r)
            for j in range(n) if rows is None else sorted(set(range(n)) & set(rows)):
                row = self.start[r] + j
                seen = [i for i in range(min(n, 64 * words if words else n)) if masks[row] >> i & 1]
                L.hold(out[row], lse[row], D.attend_row(self.q[row], values, self.base[r], seen, self.scale, self.rope))


def trees(rng, drafts):
    masks = []
    for n in drafts:
        seen = []
        for j in range(n):
            parent = rng.randint(-1, j - 1)
            seen.append((seen[parent] if parent >= 0 else 0) | 1 << j)
        masks += seen
    return masks


SIZES = [  # history, drafts, heads
    ([1000], [5], 16), ([0], [1], 1), ([0, 1, 63, 64, 65, 127, 128, 129], [1, 1, 1, 64, 63, 2, 1, 3], 8), ([300], [1], 128), ([5000], [3], 64),
    ([200, 0, 700], [16, 7, 0], 64), ([130, 64], [33, 64], 5), ([2000, 10, 1999], [4, 8, 2], 100), ([64] * 40, [1] * 40, 16), ([127], [200], 16),
    ([9000, 1], [1, 130], 3)]


@pytest.mark.parametrize("fmt", ["bf16", "mxfp4"])
@pytest.mark.parametrize("rope", [64, 0])
@pytest.mark.parametrize("base,drafts,heads", SIZES, ids=str)
def test_chains(draft, latent, base, drafts, heads, rope, fmt):
    c = Case(latent, base, drafts, heads, rope, fmt, seed=len(base) + heads)
    bad = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = c.call(draft, dev_status=bad)
    assert int(bad) == 0
    c.check(out, lse, words=None)


@pytest.mark.parametrize("fmt", ["bf16", "mxfp4"])
@pytest.mark.parametrize("base,drafts,heads", SIZES, ids=str)
def test_trees(draft, latent, base, drafts, heads, fmt):
    words = (max(drafts) + 63) // 64
    masks = trees(random.Random(heads), drafts)
    c = Case(latent, base, drafts, heads, 64, fmt, seed=heads)
    out, lse = c.call(draft, masks, words)
    c.check(out, lse, masks, words)


@pytest.mark.parametrize("base", [0, 1, 64, 200])
def test_masks_of_any_shape(draft, latent, base):
    """Masks that leave out the draft itself, that leave out everything, that see later drafts, and bits past the drafts."""
    n = 70
    rng = random.Random(base)
    masks = [rng.getrandbits(128) for _ in range(n)]
    masks[0], masks[1], masks[5], masks[69] = 0, 1 << 127, 1 << 69, (1 << 128) - 1
    c = Case(latent, [base], [n], 12, seed=base)
    out, lse = c.call(draft, masks, 2)
    c.check(out, lse, masks, 2)
    if base == 0:
        assert (out[:2] == 0).all() and torch.isinf(lse[:2]).all()
    # fewer words than drafts: those past them are not seen
    out, lse = c.call(draft, [m & (1 << 64) - 1 for m in masks], 1)
    c.check(out, lse, masks, 1)


def test_mask_words_in_a_wider_tensor(draft, latent):
    c = Case(latent, [100, 30], [6, 9], 7, seed=3)
    masks = trees(random.Random(1), c.drafts)
    wide = torch.full((15, 4), -1, dtype=torch.int64, device="cuda")
    wide[:, 1:2] = D.words(masks, 1, "cuda")
    out, lse = draft.csa_draft_attend(c.q, c.cache, c.table, c.ints(c.base), c.ints(c.start), scale=c.scale, mask=wide[:, 1:2])
    c.check(out, lse, masks, 1)


@pytest.mark.parametrize("fmt", ["bf16", "mxfp4"])
def test_rows_of_no_request_are_left(draft, latent, fmt):
    c = Case(latent, [70, 5], [3, 0], 20, fmt=fmt, spare_rows=6, seed=2)
    out, lse = torch.full((9, 20, 512), 7.0, dtype=torch.bfloat16, device="cuda"), torch.full((9, 20), 7.0, device="cuda")
    c.start = [2, 5, 5]
    c.call(draft, out=out, lse=lse)
    assert (out[:2] == 7).all() and (out[5:] == 7).all() and (lse[:2] == 7).all() and (lse[5:] == 7).all()
    c.check(out, lse, words=None, masks=[0, 0] + D.chain(3))


@pytest.mark.parametrize("pad", [16, 128])
@pytest.mark.parametrize("fmt", ["bf16", "mxfp4"])
def test_padded_pages(draft, latent, fmt, pad):
    c = Case(latent, [700, 64], [5, 9], 16, fmt=fmt, pad=pad, seed=4)
    out, lse = c.call(draft)
    c.check(out, lse, words=None)


@pytest.mark.parametrize("heads", [5, 64])
def test_strided_queries(draft, latent, heads):
    """Head-major queries, and rows with values behind them."""
    c = Case(latent, [150], [9], heads, seed=5)
    want, want_lse = c.call(draft)
    swapped = c.q.transpose(0, 1).contiguous().transpose(0, 1)
    wide = torch.full((9, heads, 600), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[..., 8:584] = c.q
    for q in (swapped, wide[..., 8:584]):
        out, lse = c.call(draft, q=q)
        assert torch.equal(out, want) and torch.equal(lse, want_lse)
    c.check(want, want_lse, words=None)


@pytest.mark.parametrize("grow,scale", [(30.0, None), (1.0, 1e-30), (1.0, 3e-39), (100.0, 1.0)])
def test_large_and_small_scores(draft, latent, grow, scale):
    """Scores of thousands (one record has all the weight; the running maximum moves) and of nothing."""
    c = Case(latent, [900], [6], 9, seed=6, grow=grow)
    c.scale = scale or c.scale
    out, lse = c.call(draft)
    c.check(out, lse, words=None)


def test_maxima_that_rise_tile_by_tile(draft, latent):
    """Each page's scores exceed the last one's by far more than 2^8: the output so far is scaled at every tile."""
    c = Case(latent, [64 * 12], [3], 16, rope=0, seed=7)
    pages = c.table[0].long()
    for p in range(13):
        records = c.cache.pages[pages[p]][:64 * 1024].view(torch.bfloat16).reshape(64, 512)
        records[records.isfinite()] *= 0.05 * (p + 1)
    c.q[:] = c.q.abs()
    for p in range(13):
        records = c.cache.pages[pages[p]][:64 * 1024].view(torch.bfloat16).reshape(64, 512)
        records.copy_(torch.where(records.isfinite(), records.abs(), records))
    c.records = c.cache.pages.reshape(-1, 1024)
    c.scale = 1.0
    out, lse = c.call(draft)
    c.check(out, lse, words=None)


def test_bad_tables_and_lengths(draft, latent):
    c = Case(latent, [200, 64], [4, 4], 6, seed=8)
    good_out, good_lse = c.call(draft)

    def run(want, **kw):
        bad = torch.zeros(1, dtype=torch.int32, device="cuda")
        out, lse = torch.full_like(good_out, 7.0), torch.full_like(good_lse, 7.0)
        args = dict(page_table=c.table, base=c.base, start=c.start)
        args.update(kw)
        draft.csa_draft_attend(c.q, c.cache, args["page_table"], c.ints(args["base"]), c.ints(args["start"]), scale=c.scale, out=out, lse=lse, dev_status=bad)
        assert int(bad) == want, kw
        return out, lse

    # a page out of range: its records are left out, the other request's answer stays
    for page in (-1, c.cache.pages.shape[0], 1 << 30):
        t = c.table.clone()
        t[0, 1] = page
        out, lse = run(1, page_table=t)
        assert torch.equal(out[4:], good_out[4:])
        v = c.values(0)
        for j in range(4):
            k = torch.cat([v[:64], v[128:200 + j + 1]])
            L.hold(out[j], lse[j], L.softmax_out(c.q[j].double(), k, k[:, :512], c.scale, 576))
    # rows' bounds
    out, lse = run(32, start=[0, 9, 9])
    assert (out == 7).all()
    out, lse = run(32, start=[4, 0, 8])
    assert (out[:0] == 7).all()
    out, lse = run(32, start=[-1, 4, 8])
    assert (out[:4] == 7).all() and torch.equal(out[4:], good_out[4:])
    # histories: below 0 is none; beyond the table is cut to it (5 pages of 64), with no draft seen
    out, lse = run(32, base=[-5, 64])
    assert torch.equal(out[4:], good_out[4:])
    full = torch.cat([c.table[:, :4], c.table[:1, :1].expand(2, 1)], 1).contiguous()
    c2 = dict(page_table=full[:, :3].contiguous())
    out, lse = run(32, base=[1 << 30, 64], **c2)
    v = c.values(0)[:192]
    for j in range(4):
        L.hold(out[j], lse[j], L.softmax_out(c.q[j].double(), v, v[:, :512], c.scale, 576))


def test_agrees_with_latent_attend(draft, latent):
    """One draft a request is an ordinary decode row."""
    c = Case(latent, [777, 64, 1], [1, 1, 1], 32, seed=9)
    out, lse = c.call(draft)
    other, other_lse = latent.csa_latent_attend(c.q, c.cache, c.table, c.ints([b + 1 for b in c.base]), scale=c.scale)
    c.check(out, lse, words=None)
    c.check(other, other_lse, words=None)


def test_nothing_to_do(draft, latent):
    c = Case(latent, [5], [0], 4, spare_rows=2)
    out, lse = torch.full((2, 4, 512), 7.0, dtype=torch.bfloat16, device="cuda"), torch.full((2, 4), 7.0, device="cuda")
    c.call(draft, out=out, lse=lse)
    assert (out == 7).all()
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    out, lse = draft.csa_draft_attend(c.q[:0], c.cache, c.table, c.ints([5]), c.ints([0, 0]), scale=1.0)
    assert out.shape == (0, 4, 512)
    out, lse = draft.csa_draft_attend(c.q, c.cache, none.reshape(0, 4), none, c.ints([0]), scale=1.0)


def test_long_histories_over_many_parts(draft, latent):
    """A history cut over all SMs and joined, and requests of very different lengths together."""
    c = Case(latent, [40000, 3, 9000], [5, 2, 11], 16, seed=10)
    masks = trees(random.Random(5), c.drafts)
    out, lse = c.call(draft, masks)
    c.check(out, lse, masks)
    again, again_lse = c.call(draft, masks)
    assert torch.equal(out, again) and torch.equal(lse, again_lse)


def test_offsets_past_32_bits(draft, latent):
    """Pages that lie beyond 4 GB of the pool."""
    pages = 60000  # of 73728 bytes: 4.4 GB
    pool = torch.empty(pages, 64 * 1152, dtype=torch.uint8, device="cuda")
    c = Case(latent, [300], [4], 16, seed=11)
    need = 5
    t = torch.full((1, need), -1, dtype=torch.int32, device="cuda")
    for p in range(need):
        t[0, p] = pages - 1 - p
        pool[pages - 1 - p] = c.cache.pages[c.table[0, p].long()]
    cache = latent.LatentCache(pool, 64, "bf16")
    out, lse = draft.csa_draft_attend(c.q, cache, t, c.ints([300]), c.ints([0, 4]), scale=c.scale)
    c.check(out, lse, words=None)


def test_bounds_that_descend_beside_rows_of_their_own(draft, latent):
    """Request 0's bounds descend: it writes nothing. Rows 0 and 1 belong to nobody; request 1 has rows 2 to 7."""
    c = Case(latent, [64, 200], [4, 6], 6, seed=12)
    c.q = c.q[:8].contiguous()
    out, lse, bad = torch.full((8, 6, 512), 7.0, dtype=torch.bfloat16, device="cuda"), torch.full((8, 6), 7.0, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    draft.csa_draft_attend(c.q, c.cache, c.table, c.ints(c.base), c.ints([4, 2, 8]), scale=c.scale, out=out, lse=lse, dev_status=bad)
    assert int(bad) == 32 and (out[:2] == 7).all() and (lse[:2] == 7).all()
    values = c.values(1)
    for j in range(6):
        L.hold(out[2 + j], lse[2 + j], D.attend_row(c.q[2 + j], values, 200, range(j + 1), c.scale, 64))


@pytest.mark.parametrize("fmt", ["bf16", "mxfp4"])
def test_scores_of_the_largest_range(draft, latent, fmt):
    """Scores q . c up to 2^125 in magnitude, both signs in a row: the softmax of a tiny scale, and with scale 1 the one record of the largest."""
    c = Case(latent, [300], [4], 5, fmt=fmt, seed=13)
    c.q[:] = 0
    c.q[..., 3] = 2.0 ** 123
    c.scale = 2.0 ** -124
    out, lse = c.call(draft)
    c.check(out, lse, words=None)
    v = c.values(0)[:, 3]
    if fmt == "bf16":  # 4-bit values tie
        c.scale = 1.0
        out, lse = c.call(draft)
        for j in range(4):
            best = int(v[:301 + j].argmax())
            second = float(v[:301 + j].sort(descending=True).values[1])
            if second < float(v[best]):
                assert torch.equal(out[j].double(), c.values(0)[best, :512].expand(5, 512))
                assert torch.allclose(lse[j].double(), v[best] * 2.0 ** 123, rtol=2 ** -20)


@pytest.mark.parametrize("fmt", ["bf16", "mxfp4"])
@pytest.mark.parametrize("base", [300, 30000])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("logit", [2.0 ** 27, 2.0 ** 30, 2.0 ** 33, 2.0 ** 36, 2.0 ** 60, 2.0 ** 126])
def test_scores_above_what_an_exponent_holds(draft, latent, logit, sign, base, fmt):
    """Scaled scores of 2^27 and more, which a tile's products with scale log2 e round by more than a softmax bears, also in requests whose parts
    are joined. The next score is 2^-8 of them less at least: the weights are 1 or 0, equal for the records of the largest."""
    c = Case(latent, [base], [3], 5, fmt=fmt, seed=14)
    c.q[:] = 0
    c.q[..., 3] = sign * 2.0 ** 100
    c.scale = logit * 2.0 ** -103  # values are below 2^3
    out, lse = c.call(draft)
    values = c.values(0)
    assert float(values[:, 3].abs().max()) < 8
    for j in range(3):
        seen = values[:base + j + 1]
        score = sign * seen[:, 3]
        best = seen[score == score.max(), :512]
        assert ((out[j].double() - best.mean(0)).abs() <= 2.1 * L.BF16_HALF * best.abs().mean(0) + 1e-30).all(), j
        want = float(score.max()) * 2.0 ** 100 * c.scale
        assert (lse[j].double() - want).abs().max() <= 2 ** -22 * abs(want)
