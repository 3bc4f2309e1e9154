"""Plain 64-bit forms of the operators of a step with drafted tokens, written from their formulas, and the
tolerances that the tests hold the kernels to.

  - A norm's factor is computed in fp32: a sum of at most 32 squares a lane and 5 steps over the lanes, each off by 2^-24,
    halved by the root, and eight operations more: NORM = (37 / 2 + 8) 2^-24 relative.
  - A cosine or sine: the angle, at most half a turn, is rounded to fp32 (pi 2^-25), the function is off by two units
    in the last place of a value up to 1 (2^-22); the products and the sum of a rotated pair take 3 2^-24 of each term, the scale another:
    TURN = 2^-22 + 6 2^-24 of |a| + |b|.
  - The result is rounded to its type once.
Attention is held to the bounds of `_latent`.
"""
from __future__ import annotations

import math

import torch

import _latent as L

F32 = L.F32_HALF
NORM, TURN = (37 / 2 + 8) * F32, 4 * F32 + 6 * F32
HALF = {torch.bfloat16: L.BF16_HALF, torch.float32: F32}


def norm(x, weight, eps):
    """x [..., dim] in fp64."""
    y = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    return y if weight is None else y * weight.double()


def rotate(x, pos, freq, pairing, scale=1.0):
    """x [n, heads, rope] in fp64 at positions [n] -> (rotated, |a| + |b| of each value's pair)."""
    n, heads, rope = x.shape
    out, size = torch.empty_like(x), torch.empty_like(x)
    for j in range(rope // 2):
        ia, ib = (2 * j, 2 * j + 1) if pairing == "adjacent" else (j, j + rope // 2)
        t = (pos.double() * freq[j].double())[:, None]
        a, b = x[..., ia], x[..., ib]
        out[..., ia] = scale * (a * torch.cos(t) - b * torch.sin(t))
        out[..., ib] = scale * (b * torch.cos(t) + a * torch.sin(t))
        size[..., ia] = size[..., ib] = abs(scale) * (a.abs() + b.abs())
    return out, size


def norm_rotate(x, weight, do_norm, eps, pos, freq, pairing, rope_first=False, scale=1.0, half=L.BF16_HALF):
    """x [n, heads, dim] -> (values, tolerances) in fp64."""
    y = norm(x.double(), weight, eps) if do_norm else x.double()
    tol = y.abs() * (NORM if do_norm else 0.0)
    rope = 0 if freq is None else 2 * freq.numel()
    if rope:
        at = slice(0, rope) if rope_first else slice(y.shape[-1] - rope, y.shape[-1])
        turned, size = rotate(y[..., at], pos, freq, pairing, scale)
        y = y.clone()
        y[..., at], tol[..., at] = turned, size * ((NORM if do_norm else 0.0) + TURN)
    return y, half * (y.abs() + tol) + tol + 1e-37


def appended(x, weight, do_norm, eps, pos, freq, pairing, fmt, scale=1.0):
    """x [n, 512 + rope] -> the values that the records stand for and their tolerances, [n, 512 + rope] in fp64."""
    x = x.double()
    y = norm(x[:, :512], weight, eps) if do_norm else x[:, :512]
    if fmt == "bf16":
        tol = L.BF16_HALF * y.abs() * (1 + NORM) + NORM * y.abs() + 1e-37
    else:
        codes, scales = L.quantise(y)
        y = L.values(torch.cat([codes, scales], 1), "mxfp4", 0)
        tol = torch.zeros_like(y)
    if x.shape[1] > 512:
        turned, t = norm_rotate(x[:, None, 512:], None, False, 0.0, pos, freq, pairing, scale=scale)
        y, tol = torch.cat([y, turned[:, 0]], 1), torch.cat([tol, t[:, 0]], 1)
    return y, tol


def freqs(rope, base=10000.0, device="cpu"):
    return (base ** (-torch.arange(0, rope, 2, dtype=torch.float64, device=device) / rope)).float()


def chain(n):
    return [(1 << (j + 1)) - 1 for j in range(n)]


def words(masks, n_words, device):
    """Bit masks (python integers) as int64 words [rows, n_words]."""
    out = []
    for m in masks:
        row = [(m >> (64 * w)) & ((1 << 64) - 1) for w in range(n_words)]
        out.append([v - (1 << 64) if v >> 63 else v for v in row])
    return torch.tensor(out, dtype=torch.int64, device=device).reshape(len(masks), n_words)


def attend_row(q, values, base, seen, scale, rope):
    """One draft's row: q [heads, 512 + rope], the request's records' values [base + drafts, 512 + rope] in fp64, the drafts that it sees."""
    at = list(range(base)) + [base + i for i in seen if base + i < values.shape[0]]
    k = values[torch.tensor(at, dtype=torch.long, device=values.device)]
    return L.softmax_out(q.double(), k, k[:, :512], scale, 512 + rope)


def commit(pool, table, base, drafts, paths, rec):
    """In place on pool [layers, pages, bytes] (host): (new lengths, pages given back)."""
    new, freed = [], []
    for r, path in enumerate(paths):
        old = pool.clone()

        def record(where, pos):
            at = pos % 64 * rec
            return where[:, table[r][pos // 64], at:at + rec]

        for k, d in enumerate(path):
            record(pool, base[r] + k).copy_(record(old, base[r] + d))
        new.append(base[r] + len(path))
        freed += table[r][math.ceil(new[-1] / 64):math.ceil((base[r] + drafts[r]) / 64)]
    return new, freed
