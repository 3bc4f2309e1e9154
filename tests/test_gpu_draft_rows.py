"""Norms with rotation, the rotating writer and the move of accepted drafts on the GPU, against their 64-bit forms."""
import math
import random
from fractions import Fraction

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


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def positions(g, n, far):
    p = torch.randint(0, far, (n,), generator=g, device="cuda").int()
    p[0] = 0
    p[-1] = far - 1
    return p


def status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def near(got, want):
    y, tol = want
    d = (got.double() - y).abs()
    assert torch.isfinite(got.double()).all()
    assert (d <= tol).all(), f"off by {d.max():.3g}, {float((d / tol).max()):.3g} of the tolerance"


# ------------------------------------------------------------------ norm and rotation

ROTATE = [  # rows, q heads, q dim, k heads, k dim, rope, pairing, rope first
    (1, 1, 64, 0, 64, 64, "adjacent", False), (64, 64, 128, 1, 128, 64, "adjacent", False), (33, 5, 192, 3, 192, 64, "halves", False),
    (7, 3, 576, 1, 64, 64, "halves", False), (5, 2, 512, 1, 576, 64, "adjacent", False), (9, 1, 64, 100, 8, 0, "adjacent", False),
    (130, 1, 128, 1, 128, 128, "halves", True), (17, 4, 256, 2, 256, 256, "halves", False), (3, 2, 1024, 1, 264, 256, "halves", False),
    (3, 2, 1016, 1, 1024, 256, "adjacent", True), (65, 7, 72, 1, 40, 32, "halves", False), (11, 128, 24, 1, 16, 16, "adjacent", True),
    (300, 1, 64, 1, 64, 64, "halves", False), (2, 128, 192, 0, 8, 64, "adjacent", False)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("case", ROTATE, ids=str)
def test_norm_and_rotation(draft, case, dtype, out):
    n, qh, qd, kh, kd, rope, pairing, first = case
    g = gen(n + qd)
    q, k = randn(g, n, qh, qd, dtype=dtype), randn(g, n, kh, kd, dtype=dtype) if kh else None
    qw, kw = 1 + 0.2 * randn(g, qd), 1 + 0.2 * randn(g, kd)
    pos, freq, bad = positions(g, n, 1 << 20), D.freqs(rope, device="cuda") if rope else None, status()
    qo, ko = draft.csa_head_norm_rotate(q, pos, freq, k=k, q_weight=qw, k_weight=kw if kh else None, eps=1e-5, pairing=pairing, rope_first=first,
                                        out_dtype=out, dev_status=bad)
    near(qo, D.norm_rotate(q, qw, True, 1e-5, pos, freq, pairing, first, half=D.HALF[out]))
    if kh:
        near(ko, D.norm_rotate(k, kw, True, 1e-5, pos, freq, pairing, first, half=D.HALF[out]))
    else:
        assert ko is None
    assert int(bad) == 0


@pytest.mark.parametrize("pairing", ["adjacent", "halves"])
@pytest.mark.parametrize("norms", [(False, False), (True, False), (False, True)])
def test_norm_of_one_tensor_and_a_scale(draft, norms, pairing):
    g = gen(3)
    q, k, pos, freq = randn(g, 40, 3, 128, dtype=torch.bfloat16), randn(g, 40, 2, 64, dtype=torch.bfloat16), positions(g, 40, 4096), D.freqs(32, device="cuda")
    qo, ko = draft.csa_head_norm_rotate(q, pos, freq, k=k, q_norm=norms[0], k_norm=norms[1], rope_scale=-1.25, pairing=pairing)
    near(qo, D.norm_rotate(q, None, norms[0], 1e-6, pos, freq, pairing, scale=-1.25))
    near(ko, D.norm_rotate(k, None, norms[1], 1e-6, pos, freq, pairing, scale=-1.25))


@pytest.mark.parametrize("pairing", ["adjacent", "halves"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("dim,rope", [(128, 64), (576, 64), (264, 256), (1024, 256)])
def test_in_place_equals_out_of_place(draft, dtype, pairing, dim, rope):
    """One head's values are another lane's partners: in place they have to be read before they are written."""
    g = gen(dim)
    pos, freq, w = positions(g, 200, 1 << 17), D.freqs(rope, device="cuda"), 1 + 0.2 * randn(g, dim)
    q = randn(g, 200, 9, dim, dtype=dtype)
    want, _ = draft.csa_head_norm_rotate(q, pos, freq, q_weight=w, pairing=pairing, out_dtype=dtype)
    got, _ = draft.csa_head_norm_rotate(q, pos, freq, q_weight=w, pairing=pairing, q_out=q)
    assert got is q and torch.equal(q, want)


def test_strided_views_and_rows_left_as_they_are(draft):
    """Queries and keys as slices of one product, the rotated part written behind absorbed values; padding rows at -1."""
    g = gen(5)
    n, heads = 21, 6
    x = randn(g, n, heads * 192 + 64 + 8, dtype=torch.bfloat16)
    q, k = x[:, :heads * 192].view(n, heads, 192)[..., 128:], x[:, heads * 192:heads * 192 + 64].unsqueeze(1)
    absorbed, keys = torch.full((n, heads, 576), 7.0, dtype=torch.bfloat16, device="cuda"), torch.full((n, 1, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    pos, freq, before = positions(g, n, 999), D.freqs(64, device="cuda"), x.clone()
    pos[3] = pos[20] = -1
    draft.csa_head_norm_rotate(q, pos, freq, k=k, q_norm=False, k_norm=False, q_out=absorbed[..., 512:], k_out=keys)
    live = pos >= 0
    assert torch.equal(x, before) and (absorbed[..., :512] == 7).all() and (absorbed[~live] == 7).all() and (keys[~live] == 5).all()
    y, tol = D.norm_rotate(q, None, False, 0.0, pos, freq, "adjacent")
    near(absorbed[live][..., 512:], (y[live], tol[live]))
    y, tol = D.norm_rotate(k, None, False, 0.0, pos, freq, "adjacent")
    near(keys[live], (y[live], tol[live]))


@pytest.mark.parametrize("pairing", ["adjacent", "halves"])
def test_far_positions(draft, pairing):
    """Angles of 2^31 radians: 2^-32 turns are 1.5e-9 of a unit, far below TURN. The 64-bit form's own angle is off by 2^31 2^-53."""
    g = gen(8)
    pos = torch.tensor([0, 1, 2, 65537, (1 << 24) + 1, (1 << 30) + 7, (1 << 31) - 1], dtype=torch.int32, device="cuda")
    freq = torch.tensor([1.0, 0.9999, 0.3, 1e-4, 1e-9, 0.0, -0.7, 6.2831855], dtype=torch.float32, device="cuda")
    q = randn(g, len(pos), 2, 16)
    out, _ = draft.csa_head_norm_rotate(q, pos, freq, q_norm=False, pairing=pairing, out_dtype=torch.float32)
    y, tol = D.norm_rotate(q, None, False, 0.0, pos, freq, pairing, half=D.F32)
    near(out, (y, tol + 1e-6 * 2 ** -1))


PI = Fraction("3.14159265358979323846264338327950288419716939937510582097494459")


def exact_turn(pos, freq):
    """cos and sin of pos * freq from whole numbers: the angle's turns modulo 1 before anything is rounded."""
    turns = Fraction(pos) * Fraction(freq) / (2 * PI) % 1
    return math.cos(2 * math.pi * float(turns)), math.sin(2 * math.pi * float(turns))


@pytest.mark.parametrize("pairing", ["adjacent", "halves"])
def test_large_frequencies(draft, latent, pairing):
    """Up to 2^10 radians a token, at positions up to 2^31 - 1; in the heads, and in the writer's records."""
    g = gen(16)
    at = [0, 1, 3, 4097, (1 << 24) + 1, (1 << 31) - 2, (1 << 31) - 1]
    f = [1024.0, -1024.0, 1023.9999, 777.125, -100.7, 6.2831855, 2.0 ** -140, 0.5] * 4
    pos, freq = torch.tensor(at, dtype=torch.int32, device="cuda"), torch.tensor(f, dtype=torch.float32, device="cuda")
    q = randn(g, len(at), 2, 64)
    turned, size = torch.empty_like(q, dtype=torch.float64), torch.empty_like(q, dtype=torch.float64)
    for j in range(32):
        ia, ib = (2 * j, 2 * j + 1) if pairing == "adjacent" else (j, j + 32)
        a, b = q[..., ia].double(), q[..., ib].double()
        turn = torch.tensor([exact_turn(p, float(freq[j])) for p in at], dtype=torch.float64, device="cuda")[:, None]
        turned[..., ia], turned[..., ib] = a * turn[..., 0] - b * turn[..., 1], b * turn[..., 0] + a * turn[..., 1]
        size[..., ia] = size[..., ib] = a.abs() + b.abs()
    tol = D.TURN * size
    out, _ = draft.csa_head_norm_rotate(q, pos, freq, q_norm=False, pairing=pairing, out_dtype=torch.float32)
    near(out, (turned, tol + D.F32 * (turned.abs() + tol) + 1e-37))
    x = torch.cat([torch.ones(len(at), 512, device="cuda"), q[:, 0]], 1)
    cache, slots = latent.LatentCache.empty(1, 64, "bf16"), torch.arange(len(at), device="cuda")
    draft.csa_latent_append(x, slots, pos, cache, freq, norm=False, pairing=pairing)
    near(read_back(cache, slots, "bf16", 64)[:, 512:], (turned[:, 0], (tol + L.BF16_HALF * (turned.abs() + tol) + 1e-37)[:, 0]))


@pytest.mark.parametrize("scale", [1e-30, 1e-18, 1e18, 1e30, 3e37])
@pytest.mark.parametrize("dim", [64, 192, 1024])
def test_squares_outside_fp32(draft, dim, scale):
    """Heads whose squares overflow or vanish in fp32, beside ordinary ones; eps as small as their squares, or none."""
    g = gen(9)
    x = randn(g, 10, 3, dim)
    x[:, 1] *= scale
    for eps in (1e-6, 0.0):
        got, _ = draft.csa_head_norm_rotate(x, None, None, eps=eps, out_dtype=torch.float32)
        near(got, D.norm_rotate(x, None, True, eps, None, None, "adjacent", half=D.F32))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("pairing", ["adjacent", "halves"])
@pytest.mark.parametrize("scale", [1e-39, 3e-40, 2.0 ** -126, 2.0 ** -120, 1e-34, 2.0 ** 125, 3e38])
def test_factors_outside_fp32(draft, scale, pairing, dtype):
    """Heads of subnormal values, whose factor is above fp32's largest number, and of the largest, whose factor is subnormal. The values are
    rounded to the input's type before the 64-bit form sees them. One head has a single value that is not 0, the smallest of all."""
    g = gen(12)
    x = randn(g, 10, 3, 128)
    x = ((torch.sign(x) if scale > 1e38 else x.clamp(-7, 7)) * scale).to(dtype)
    x[:, 1] = 0
    x[:, 1, 100] = 2.0 ** (-149 if dtype == torch.float32 else -133)
    assert x.double().isfinite().all() and (x[:, 0] != 0).any(-1).all()
    pos, freq, w = positions(g, 10, 1 << 17), D.freqs(64, device="cuda"), 1 + 0.2 * randn(g, 128)
    got, _ = draft.csa_head_norm_rotate(x, pos, freq, q_weight=w, eps=0.0, pairing=pairing, out_dtype=torch.float32)
    near(got, D.norm_rotate(x, w, True, 0.0, pos, freq, pairing, half=D.F32))
    in_place, _ = draft.csa_head_norm_rotate(x, pos, freq, q_weight=w, eps=0.0, pairing=pairing, q_out=x)
    assert in_place is x and torch.equal(x, got.to(dtype))


@pytest.mark.parametrize("pairing", ["adjacent", "halves"])
@pytest.mark.parametrize("top", [2.0 ** 20, 2.0 ** 40, 2.0 ** 126])
def test_subnormal_values_with_large_weights(draft, latent, top, pairing):
    """Values that become fp32's subnormal numbers when they are normed, and that their weights lift again: 2^-150 of each is lost, times its
    weight (below 1.5 top); a rotated value is made of two. In the heads and in records of bf16."""
    g = gen(14)
    x, pos, freq = randn(g, 128, 576), positions(g, 128, 1 << 17), D.freqs(64, device="cuda")
    x[:, 32:512] *= 2.0 ** -138
    w = top * (1 + 0.5 * torch.rand(512, generator=g, device="cuda"))
    w[:32] = 1
    lost = 2 * 2.0 ** -150 * 1.5 * top
    got, _ = draft.csa_head_norm_rotate(x[:, None, :512], pos, freq, q_weight=w, eps=1e-6, pairing=pairing, out_dtype=torch.float32)
    y, tol = D.norm_rotate(x[:, None, :512], w, True, 1e-6, pos, freq, pairing, half=D.F32)
    near(got, (y, tol + lost))
    cache, slots, bad = latent.LatentCache.empty(2, 64, "bf16"), torch.arange(128, device="cuda"), status()
    draft.csa_latent_append(x, slots, pos, cache, freq, weight=w, eps=1e-6, pairing=pairing, dev_status=bad)
    y, tol = D.appended(x, w, True, 1e-6, pos, freq, pairing, "bf16")
    near(read_back(cache, slots, "bf16", 64), (y, tol + lost * (1 + L.BF16_HALF)))
    assert int(bad) == 0


def test_not_finite_and_zero_heads(draft):
    """A NaN stays in its head; an infinity makes its head's others 0; zeros are 0 with an eps and NaN without."""
    x = torch.ones(4, 3, 128, device="cuda")
    x[0, 0, 5], x[1, 1, 9], x[2, 2] = float("nan"), float("inf"), 0.0
    got, _ = draft.csa_head_norm_rotate(x, None, None, eps=1e-6, out_dtype=torch.float32)
    assert got[0, 0].isnan().all() and got[0, 1:].isfinite().all()
    assert got[1, 1, 9].isnan() and (got[1, 1, :9] == 0).all() and (got[1, 1, 10:] == 0).all() and got[1, 0].isfinite().all()
    assert (got[2, 2] == 0).all()
    got, _ = draft.csa_head_norm_rotate(x, None, None, eps=0.0, out_dtype=torch.float32)
    assert got[2, 2].isnan().all() and got[2, :2].isfinite().all()


def test_bad_positions_leave_their_rows(draft):
    q = torch.ones(5, 2, 64, dtype=torch.bfloat16, device="cuda")
    out, bad = torch.full_like(q, 3.0), status()
    draft.csa_head_norm_rotate(q, torch.tensor([0, -2, 4, -1, 9], dtype=torch.int32, device="cuda"), D.freqs(64, device="cuda"), q_out=out, dev_status=bad)
    assert int(bad) == 32 and (out[1] == 3).all() and (out[3] == 3).all() and not (out[0] == 3).any()


def test_nothing_to_do(draft):
    freq = D.freqs(64, device="cuda")
    q, k = draft.csa_head_norm_rotate(torch.empty(0, 4, 64, device="cuda"), torch.empty(0, dtype=torch.int32, device="cuda"), freq)
    assert q.shape == (0, 4, 64) and k is None
    one = torch.ones(3, 2, 64, device="cuda")
    q, k = draft.csa_head_norm_rotate(one[:, :0], torch.zeros(3, dtype=torch.int32, device="cuda"), freq, k=one, k_norm=False, out_dtype=torch.float32)
    assert q.shape == (3, 0, 64) and torch.equal(k, one)


# ------------------------------------------------------------------ the rotating writer

def read_back(cache, slots, fmt, rope):
    records = cache.pages[:, :64 * cache.record_bytes].reshape(-1, cache.record_bytes)
    return L.values(records[slots], fmt, rope)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("fmt", ["bf16", "mxfp4"])
@pytest.mark.parametrize("rope,pairing", [(0, "adjacent"), (64, "adjacent"), (64, "halves")])
@pytest.mark.parametrize("n", [1, 7, 64, 1000])
def test_append(draft, latent, n, rope, pairing, fmt, dtype):
    g = gen(n + rope)
    cache = latent.LatentCache.empty(n // 64 + 3, rope, fmt)
    cache.pages.fill_(0xA5)
    untouched = cache.pages.clone()
    wide = randn(g, n, 512 + rope + 8) * torch.exp2(torch.randint(-6, 7, (n, 1), generator=g, device="cuda").float())
    x = wide.to(dtype)[:, :512 + rope]
    slots = torch.randperm((n // 64 + 3) * 64, generator=g, device="cuda")[:n]
    pos, freq, w, bad = positions(g, n, 1 << 20), D.freqs(64, device="cuda"), 1 + 0.2 * randn(g, 512), status()
    draft.csa_latent_append(x, slots, pos, cache, freq, weight=w, eps=1e-5, pairing=pairing, dev_status=bad)
    near(read_back(cache, slots, fmt, rope), D.appended(x, w, True, 1e-5, pos, freq, pairing, fmt))
    assert int(bad) == 0
    rest = torch.ones(cache.pages.shape[0] * 64, dtype=torch.bool, device="cuda")
    rest[slots] = False
    assert torch.equal(cache.pages.reshape(-1, cache.record_bytes)[rest], untouched.reshape(-1, cache.record_bytes)[rest])


@pytest.mark.parametrize("fmt", ["bf16", "mxfp4"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_append_without_norm_at_position_0_is_the_writer(draft, latent, dtype, fmt):
    g = gen(1)
    a, b = latent.LatentCache.empty(3, 64, fmt), latent.LatentCache.empty(3, 64, fmt)
    a.pages.zero_(), b.pages.zero_()
    x, slots = randn(g, 150, 576, dtype=dtype), torch.randperm(192, generator=g, device="cuda")[:150]
    draft.csa_latent_append(x, slots, torch.zeros(150, dtype=torch.int32, device="cuda"), a, D.freqs(64, device="cuda"), norm=False)
    latent.csa_latent_write(x, slots, b)
    assert torch.equal(a.pages, b.pages)


def test_four_bit_codes_next_to_their_borders(draft, latent):
    """Normed values that lie on a border between two codes, or between two exponents, to within a few 2^-24: the codes are those of the
    exact norm. Rows of ones and one larger value: with weight b / (1 / sqrt(mean)) values sit at b times a power of two."""
    n = 4096
    g = gen(2)
    x = torch.sign(randn(g, n, 512)) * (1 + torch.randint(0, 3, (n, 512), generator=g, device="cuda").float())
    border = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 4.0], dtype=torch.float64, device="cuda")
    r = 1.0 / torch.sqrt((x[0].double() ** 2).mean() + 1e-6)
    w = (border[torch.arange(512, device="cuda") % 8] / r).float()  # row 0 lands on borders to 2^-24; the others near theirs
    x[1::2] = x[0]
    x[1::2] *= (1 + torch.randint(-4, 5, (n // 2, 1), generator=g, device="cuda").float() * 2 ** -22)
    cache = latent.LatentCache.empty(n // 64, 0, "mxfp4")
    slots = torch.arange(n, device="cuda")
    draft.csa_latent_append(x, slots, None, cache, None, weight=w, eps=1e-6)
    want, _ = D.appended(x, w, True, 1e-6, None, None, "adjacent", "mxfp4")
    assert torch.equal(read_back(cache, slots, "mxfp4", 0), want)


@pytest.mark.parametrize("top", [2.0 ** 20, 2.0 ** 40, 2.0 ** 126])
def test_four_bit_codes_of_subnormal_values_with_large_weights(draft, latent, top):
    """Values that become fp32's subnormal numbers, with few bits, when they are normed, and that their weights lift again."""
    n = 256
    g = gen(8)
    x = randn(g, n, 512)
    x[:, 32:] *= 2.0 ** -138
    w = top * (1 + 0.5 * torch.rand(512, generator=g, device="cuda"))
    w[:32] = 1
    cache, slots, bad = latent.LatentCache.empty(n // 64, 0, "mxfp4"), torch.arange(n, device="cuda"), status()
    draft.csa_latent_append(x, slots, None, cache, None, weight=w, eps=1e-6, dev_status=bad)
    want, _ = D.appended(x, w, True, 1e-6, None, None, "adjacent", "mxfp4")
    assert torch.equal(read_back(cache, slots, "mxfp4", 0), want) and int(bad) == 0


@pytest.mark.parametrize("fmt", ["bf16", "mxfp4"])
@pytest.mark.parametrize("scale", [1e-38, 1e-25, 1e-12, 1e12, 1e25, 3e37])
def test_append_squares_outside_fp32(draft, latent, scale, fmt):
    g = gen(4)
    x = randn(g, 70, 512) * scale
    slots, cache = torch.arange(70, device="cuda"), latent.LatentCache.empty(2, 0, fmt)
    for eps in (1e-6, 1e-37):
        draft.csa_latent_append(x, slots, None, cache, None, eps=eps)
        near(read_back(cache, slots, fmt, 0), D.appended(x, None, True, eps, None, None, "adjacent", fmt))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("fmt", ["bf16", "mxfp4"])
@pytest.mark.parametrize("scale", [1e-39, 3e-40, 2.0 ** -126, 2.0 ** -120, 1e-34, 2.0 ** 125, 3e38])
def test_append_factors_outside_fp32(draft, latent, scale, fmt, dtype):
    """Rows of subnormal values without an eps, and of the largest; a row with a single value, the smallest of all."""
    g = gen(13)
    x = randn(g, 70, 512)
    x = ((torch.sign(x) if scale > 1e38 else x.clamp(-7, 7)) * scale).to(dtype)
    x[7] = 0
    x[7, 300] = 2.0 ** (-149 if dtype == torch.float32 else -133)
    slots, cache, bad, w = torch.arange(70, device="cuda"), latent.LatentCache.empty(2, 0, fmt), status(), 1 + 0.2 * randn(g, 512)
    cache.pages.fill_(0x77)
    draft.csa_latent_append(x, slots, None, cache, None, weight=w, eps=0.0, dev_status=bad)
    near(read_back(cache, slots, fmt, 0), D.appended(x, w, True, 0.0, None, None, "adjacent", fmt))
    assert int(bad) == 0


@pytest.mark.parametrize("fmt", ["bf16", "mxfp4"])
def test_append_bad_rows_are_left_out(draft, latent, fmt):
    g = gen(6)
    cache = latent.LatentCache.empty(2, 64, fmt)
    cache.pages.fill_(0x11)
    x, before = randn(g, 8, 576), cache.pages.clone()
    x[1, 100], x[2, 570], x[3, 3] = float("nan"), float("inf"), float("-inf")
    slots = torch.tensor([0, 1, 2, 3, -1, 128, -7, 5], device="cuda")
    pos = torch.tensor([3, 3, 3, 3, -5, 3, 3, -1], dtype=torch.int32, device="cuda")
    for rows, flag in (([0], 0), ([1], 4), ([2], 4), ([3], 4), ([4], 0), ([5], 1), ([6], 1), ([7], 32)):
        bad = status()
        draft.csa_latent_append(x[rows], slots[rows], pos[rows], cache, D.freqs(64, device="cuda"), dev_status=bad)
        assert int(bad) == flag, rows
    records = cache.pages.reshape(-1, cache.record_bytes)
    assert torch.equal(records[1:], before.reshape(-1, cache.record_bytes)[1:]) and not torch.equal(records[0], before.reshape(-1, cache.record_bytes)[0])


# ------------------------------------------------------------------ accepted drafts

def commit_case(rng, requests, most, layers, fmt, rope, spare=5):
    base = [rng.choice([0, 1, 63, 64, rng.randint(0, 200)]) for _ in range(requests)]
    drafts = [rng.randint(0, most) for _ in range(requests)]
    paths = [sorted(rng.sample(range(n), rng.randint(0, n))) for n in drafts]
    width = max(1, max((b + n + 63) // 64 for b, n in zip(base, drafts)))
    pages = sum((b + n + 63) // 64 for b, n in zip(base, drafts)) + spare
    order = list(range(pages))
    rng.shuffle(order)
    table = [[order.pop() if p < (b + n + 63) // 64 else -1 for p in range(width)] for b, n in zip(base, drafts)]
    rec = L.record_bytes(fmt, rope)
    pool = torch.randint(0, 256, (layers, pages, 64 * rec), dtype=torch.uint8, generator=torch.Generator().manual_seed(rng.randrange(1 << 30)))
    return base, drafts, paths, table, pool, rec


def ints(v, shape=None):
    t = torch.tensor(v, dtype=torch.int32, device="cuda")
    return t if shape is None else t.reshape(shape)


@pytest.mark.parametrize("fmt,rope", [("bf16", 64), ("bf16", 0), ("mxfp4", 64), ("mxfp4", 0)])
@pytest.mark.parametrize("requests,most,layers", [(1, 1, 1), (3, 9, 1), (7, 40, 5), (300, 5, 1), (2, 300, 3), (5, 16, 37), (900, 3, 1)])
def test_commit(draft, requests, most, layers, fmt, rope):
    rng = random.Random(requests * most + layers)
    base, drafts, paths, table, pool, rec = commit_case(rng, requests, most, layers, fmt, rope)
    cache = draft.LayeredCache(pool.cuda(), rope, fmt)
    wide = max(1, max(len(p) for p in paths))
    bad, t = status(), ints(table)
    new, freed = D.commit(pool, table, base, drafts, paths, rec)
    r = draft.csa_draft_commit(cache, t, ints(base), ints(drafts), ints([p + [-9] * (wide - len(p)) for p in paths]), ints([len(p) for p in paths]),
                               room=len(freed) + 3, dev_status=bad)
    assert torch.equal(cache.pages.cpu(), pool) and r.new_len.tolist() == new
    assert r.n_freed.tolist() == [len(freed)] and r.freed.tolist() == freed + [-1] * 3
    assert int(bad) == 0 and torch.equal(t, ints(table))


def test_commit_of_one_cache_and_padded_pages(draft, latent):
    rng = random.Random(4)
    base, drafts, paths, table, pool, rec = commit_case(rng, 6, 20, 1, "mxfp4", 64)
    padded = torch.zeros(pool.shape[1], 64 * rec + 48, dtype=torch.uint8, device="cuda")
    padded[:, :64 * rec] = pool[0].cuda()
    cache = latent.LatentCache(padded, 64, "mxfp4")
    new, freed = D.commit(pool, table, base, drafts, paths, rec)
    wide = max(1, max(len(p) for p in paths))
    r = draft.csa_draft_commit(cache, ints(table), ints(base), ints(drafts), ints([p + [0] * (wide - len(p)) for p in paths]), ints([len(p) for p in paths]))
    assert torch.equal(padded[:, :64 * rec].cpu(), pool[0]) and not padded[:, 64 * rec:].any()
    assert r.new_len.tolist() == new and r.freed[:len(freed)].tolist() == freed and (r.freed[len(freed):] == -1).all()


@pytest.mark.parametrize("fmt,rope", [("bf16", 64), ("mxfp4", 0)])
def test_commit_of_layers_within_each_page(draft, fmt, rope):
    """A pool whose pages hold every layer's records one after the other: layers are closer together than pages."""
    rng = random.Random(6)
    base, drafts, paths, table, pool, rec = commit_case(rng, 9, 12, 4, fmt, rope)
    pages = pool.transpose(0, 1).contiguous().cuda().transpose(0, 1)
    cache = draft.LayeredCache(pages, rope, fmt)
    assert cache.layer_stride == 64 * rec and cache.args.page_stride_bytes == 4 * 64 * rec
    new, freed = D.commit(pool, table, base, drafts, paths, rec)
    wide = max(1, max(len(p) for p in paths))
    r = draft.csa_draft_commit(cache, ints(table), ints(base), ints(drafts), ints([p + [0] * (wide - len(p)) for p in paths]), ints([len(p) for p in paths]))
    assert torch.equal(pages.cpu(), pool) and r.new_len.tolist() == new and r.freed[:len(freed)].tolist() == freed


def test_commit_of_the_most_requests(draft):
    """16384 of them, one layer, every eleventh refused."""
    n, rng = draft.COMMIT_MAX_REQ, random.Random(7)
    base, drafts = [rng.randint(0, 100) for _ in range(n)], [rng.randint(0, 4) for _ in range(n)]
    paths = [sorted(rng.sample(range(d), rng.randint(0, d))) for d in drafts]
    table = [[2 * r, 2 * r + 1] for r in range(n)]
    pool = torch.randint(0, 256, (1, 2 * n, 64 * 272), dtype=torch.uint8, generator=torch.Generator().manual_seed(8))
    lens = [len(p) for p in paths]
    for r in range(0, n, 11):
        lens[r] = drafts[r] + 1
    cache, bad = draft.LayeredCache(pool.cuda(), 0, "mxfp4"), status()
    r = draft.csa_draft_commit(cache, ints(table), ints(base), ints(drafts), ints([p + [0] * (5 - len(p)) for p in paths]), ints(lens), dev_status=bad)
    freed, new = [], []
    for i in range(n):
        ok = i % 11 != 0
        new.append(base[i] + (len(paths[i]) if ok else 0))
        if ok:
            freed += table[i][-(-new[-1] // 64):-(-(base[i] + drafts[i]) // 64)]
            for k, d in enumerate(paths[i]):  # ascending, and never behind its place: in order, in place
                to, by = base[i] + k, base[i] + d
                pool[0, table[i][to // 64], to % 64 * 272:(to % 64 + 1) * 272] = pool[0, table[i][by // 64], by % 64 * 272:(by % 64 + 1) * 272]
    assert int(bad) == 32 and r.new_len.tolist() == new and r.n_freed.tolist() == [len(freed)] and r.freed[:len(freed)].tolist() == freed
    assert torch.equal(cache.pages.cpu(), pool)


def test_commit_bad_requests_are_left_as_they_are(draft):
    """Each of the refused requests beside a good one, whose records move."""
    pool = torch.randint(0, 256, (1, 8, 64 * 400), dtype=torch.uint8, generator=torch.Generator().manual_seed(1))
    good = [0, 1, 4, -1]
    #          table, base, drafts, path, length, flag
    cases = [([2, 3, -1, -1], -1, 5, [0, 1], 2, 32), ([2, 3, -1, -1], 250, 7, [0, 3], 2, 32), ([2, 3, -1, -1], 5, 5, [0, 5], 2, 32),
             ([2, 3, -1, -1], 5, 5, [1, 1], 2, 32), ([2, 3, -1, -1], 5, 5, [2, 1], 2, 32), ([2, 3, -1, -1], 5, 5, [-1, 1], 2, 32),
             ([2, 3, -1, -1], 5, 1, [0, 1], 2, 32), ([2, 3, -1, -1], 5, 5, [0, 1], 3, 32), ([2, 3, -1, -1], 5, 5, [0, 1], -1, 32),
             ([2, 3, -1, -1], 5, -1, [0, 1], 0, 32), ([2, 8, -1, -1], 60, 9, [0, 7], 2, 1), ([2, -1, -1, -1], 60, 9, [0, 1], 2, 1),
             ([-3, 3, -1, -1], 62, 9, [1, 7], 2, 1)]
    for table, base, drafts, path, length, flag in cases:
        cache, bad = draft.LayeredCache(pool.cuda(), 64, "mxfp4"), status()
        want = pool.clone()
        new, freed = D.commit(want, [good], [60], [70], [[1, 4]], 400)
        r = draft.csa_draft_commit(cache, ints([good, table]), ints([60, base]), ints([70, drafts]), ints([[1, 4], path]), ints([2, length]), room=4,
                                   dev_status=bad)
        assert int(bad) == flag and torch.equal(cache.pages.cpu(), want), (table, base, drafts, path, length)
        assert r.new_len.tolist() == new + [base] and r.n_freed.tolist() == [len(freed)] and r.freed.tolist() == (freed + [-1] * 4)[:4]


def test_commit_more_pages_than_room(draft):
    pool, bad = torch.zeros(1, 9, 64 * 272, dtype=torch.uint8, device="cuda"), status()
    cache = draft.LayeredCache(pool, 0, "mxfp4")
    r = draft.csa_draft_commit(cache, ints([[0, 1, 2, 3], [4, 5, 6, 7]]), ints([0, 64]), ints([256, 130]), ints([[0], [0]]), ints([0, 1]), room=3, dev_status=bad)
    assert r.n_freed.tolist() == [6] and r.freed.tolist() == [0, 1, 2] and int(bad) == 128 and r.new_len.tolist() == [0, 65]
    r = draft.csa_draft_commit(cache, ints([[0, 1, 2, 3]]), ints([0]), ints([256]), torch.zeros(1, 0, dtype=torch.int32, device="cuda"), ints([0]), room=0)
    assert r.n_freed.tolist() == [4] and r.freed.numel() == 0


def test_commit_no_requests(draft):
    cache = draft.LayeredCache.empty(2, 3, 0, "mxfp4")
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    r = draft.csa_draft_commit(cache, none.reshape(0, 4), none, none, none.reshape(0, 2), none, room=2)
    assert r.n_freed.tolist() == [0] and r.freed.tolist() == [-1, -1] and r.new_len.numel() == 0
