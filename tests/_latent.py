"""Plain 64-bit forms of the latent-cache operators, written from their formulas,
and the tolerances that the tests hold the kernels to.

A rounding to a type is off by at most half a step of it: 2^-8 relative for bf16,
2^-24 for fp32. Of an attention output o = sum_n p_n v_n (p the softmax):
  - each p_n may be rounded to bf16 once before it meets v_n:   2^-8 sum p |v|
  - the output is rounded to bf16 once:                          2^-8 |o|
  - scores, exponentials, sums and products are fp32. A score of n products is off by
    at most n 2^-24 sum |q c| (products of bf16 are exact in fp32), which moves p by that
    factor; the exponential, its argument's scaling and the sums add a few 2^-24 of |s| and
    of p. E below bounds the shift of a score; p is off by about 2 E relative.
  - lse is off by E, and by a few 2^-24 of itself.
"""
from __future__ import annotations

import math

import torch

LATENT, PAGE = 512, 64
BF16_HALF, F32_HALF = torch.finfo(torch.bfloat16).eps / 2, torch.finfo(torch.float32).eps / 2
E2M1 = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)


def record_bytes(fmt, rope):
    return 2 * (LATENT + rope) if fmt == "bf16" else LATENT // 2 + LATENT // 32 + 2 * rope


def quantise(x):
    """fp64 rows [n, 512] -> (code bytes [n, 256], scale bytes [n, 16]); by search of the nearest value."""
    b = x.reshape(x.shape[0], 16, 32)
    amax = b.abs().amax(-1)
    # frexp: amax = f 2^e, f in [1/2, 1), exact where a rounded logarithm can fall below an exact power of two
    e = torch.where(amax > 0, torch.frexp(amax)[1].double() - 3, torch.full_like(amax, -127)).clamp(min=-127)
    y = (b / torch.exp2(e)[..., None])
    grid = E2M1.to(x.device)
    d = (y.abs().clamp(max=6.0)[..., None] - grid).abs()
    # nearest, ties to the even code: an odd code loses a tie by being moved a little away
    odd = (torch.arange(8, device=x.device) % 2).double() * 1e-12
    code = (d + odd).argmin(-1) | (torch.signbit(y).long() << 3)
    code = code.reshape(x.shape[0], 256, 2)
    return (code[..., 0] | (code[..., 1] << 4)).to(torch.uint8), (e + 127).to(torch.uint8)


def make_records(x, fmt, rope):
    """fp32 or bf16 rows [n, 512 + rope] -> record bytes [n, rec]."""
    tail = x.to(torch.bfloat16)
    if fmt == "bf16":
        return tail.contiguous().view(torch.uint8).reshape(x.shape[0], -1)
    codes, scales = quantise(x[:, :LATENT].double())
    return torch.cat([codes, scales, tail[:, LATENT:].contiguous().view(torch.uint8).reshape(x.shape[0], -1)], 1)


def values(records, fmt, rope):
    """Record bytes [n, rec] -> fp64 values [n, 512 + rope]."""
    if fmt == "bf16":
        return records.contiguous().view(torch.bfloat16).double()
    codes = torch.stack([records[:, :256] & 15, records[:, :256] >> 4], -1).reshape(records.shape[0], LATENT).long()
    v = E2M1.to(records.device)[codes & 7] * (1.0 - 2.0 * (codes >> 3).double())
    s = torch.exp2(records[:, 256:272].double() - 127)
    s = torch.where(records[:, 256:272] == 255, torch.full_like(s, math.nan), s)
    v = v * s.repeat_interleave(32, 1)
    if not rope:
        return v
    return torch.cat([v, records[:, 272:].contiguous().view(torch.bfloat16).double().reshape(-1, rope)], 1)


def softmax_out(q, k, v, scale, products):
    """One row and head group: q [h, d], k [n, d], v [n, dv] in fp64 ->
    (out [h, dv], lse [h], bound on |out error| [h, dv], bound on |lse error| [h])."""
    h, n = q.shape[0], k.shape[0]
    if n == 0:
        z = torch.zeros(h, v.shape[1], dtype=torch.float64, device=q.device)
        return z, torch.full((h,), -math.inf, dtype=torch.float64, device=q.device), z, torch.zeros(h, dtype=torch.float64, device=q.device)
    s = q @ k.t() * scale
    lse = torch.logsumexp(s, 1)
    p = torch.exp(s - lse[:, None])
    out = p @ v
    size = q.abs() @ k.abs().t() * scale
    e = ((products + 4) * F32_HALF * size).amax(1) + 16 * F32_HALF * (1 + s.abs().amax(1))
    weight = p @ v.abs()
    tol_lse = e + 16 * F32_HALF * (1 + lse.abs())
    tol_out = BF16_HALF * out.abs() + (BF16_HALF * 1.01 + 2 * e[:, None] + (n + 8) * F32_HALF) * weight + 1e-37
    return out, lse, tol_out, tol_lse


def hold(got_out, got_lse, want):
    """Asserts one row's outputs [h, dv], [h] against softmax_out's answer."""
    out, lse, tol_out, tol_lse = want
    g, gl = got_out.double(), got_lse.double()
    empty = torch.isinf(lse)
    assert torch.equal(torch.isinf(gl), empty), (gl, lse)
    assert torch.isfinite(g).all()
    d = (g - out).abs()
    assert (d <= tol_out).all(), f"out: off by {d.max():.3g}, {float((d / tol_out.clamp(min=1e-300)).max()):.3g} of the tolerance"
    dl = torch.where(empty, torch.zeros_like(lse), (gl - lse).abs())
    assert (dl <= tol_lse).all(), f"lse: off by {dl.max():.3g}"


def tables(old, new, table, free, n_rows):
    """csa_build_tables on host lists (in-range lengths, enough free pages)."""
    req, pos, slot, start, kv, taken = [], [], [], [0], [0], 0
    for r, (a, b) in enumerate(zip(old, new)):
        for p in range(-(-a // PAGE), -(-(a + b) // PAGE)):
            table[r][p] = free[taken]
            taken += 1
        for n in range(a, a + b):
            req.append(r)
            pos.append(n)
            slot.append(table[r][n // PAGE] * PAGE + n % PAGE)
        start.append(start[-1] + b)
        kv.append(kv[-1] + a + b)
    blank = n_rows - len(req)
    return dict(row_req=req + [0] * blank, row_pos=pos + [-1] * blank, row_len=[p + 1 for p in pos] + [0] * blank,
                row_slot=slot + [-1] * blank, row_start=start, kv_start=kv, taken=[taken])
