"""Measured cases of a step with drafted tokens over the latent cache: norms and rotation of queries and keys,
latents normed, rotated and stored in the paged cache, attention of a tree of drafts over it, and the accepted drafts' records
moved to the front.

`run` computes an operator in elementary torch operations, or, where `own` is set, calls the library.
"""
import math
import random

import torch

own = False

PAGE = 64          # records a page
LATENT = 512       # latent values of a record: keys and values
BF16, MXFP4 = "bf16", "mxfp4"
EPS = 1e-6
DTYPE = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # the indexer's queries and keys of one decode step: 64 query heads, one key head
        dict(name="rotate_decode", op="rotate", rows=64, q_heads=64, k_heads=1, dim=128, rope=64, pairing="adjacent", source="bf16", far=131071),
        # the expanded attention's queries of a prompt chunk, a norm for each head
        dict(name="rotate_chunk", op="rotate", rows=16384, q_heads=16, k_heads=1, dim=192, rope=64, pairing="adjacent", source="bf16", far=32767),
        # few heads of a sharded layer out of an fp32 product, grouped keys, far positions
        dict(name="rotate_ragged_fp32", op="rotate", rows=1021, q_heads=5, k_heads=3, dim=576, rope=64, pairing="halves", source="fp32", far=1048575),
        # the latents of one decode step of 64 requests
        dict(name="append_decode", op="append", rows=64, rope=64, fmt=BF16, source="bf16", pairing="adjacent", far=131071, back=False),
        # the latents of a prompt, a slice of the projection's product
        dict(name="append_prompt", op="append", rows=16381, rope=64, fmt=BF16, source="bf16", pairing="halves", far=1048575, back=False),
        # a wave of prompts, fp32 out of the projection, stored in 4 bits and read back for the expansion
        dict(name="append_read_mxfp4", op="append", rows=65537, rope=64, fmt=MXFP4, source="fp32", pairing="adjacent", far=65537, back=True),
        # five drafts of one short request, few heads of a sharded layer: latency
        dict(name="verify_one", op="verify", requests=1, lo=1000, hi=1000, drafts_lo=5, drafts_hi=5, heads=16, rope=64, fmt=BF16, tree=True),
        # trees of 16 drafts of two very long requests, all heads on one GPU
        dict(name="verify_long", op="verify", requests=2, lo=65536, hi=131072, drafts_lo=16, drafts_hi=16, heads=64, rope=64, fmt=BF16, tree=True),
        # a batch of requests with 1 to 8 drafts in a chain, the heads of a sharded layer
        dict(name="verify_batch", op="verify", requests=32, lo=8192, hi=32768, drafts_lo=1, drafts_hi=8, heads=16, rope=64, fmt=BF16, tree=False),
        # trees of up to 13 drafts over a cache held in 4 bits
        dict(name="verify_4bit", op="verify", requests=16, lo=7001, hi=16384, drafts_lo=3, drafts_hi=13, heads=64, rope=64, fmt=MXFP4, tree=True),
        # one layer's cache after a step of a small batch
        dict(name="commit_step", op="commit", requests=8, layers=1, drafts_lo=5, drafts_hi=16, rope=64, fmt=MXFP4),
        # every layer's cache of a batch after a step
        dict(name="commit_layers", op="commit", requests=48, layers=24, drafts_lo=16, drafts_hi=48, rope=64, fmt=BF16),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    while True:
        c = _draw(rng)
        w = work(c)
        if w["bytes"] <= 8e8 and w["flops"] <= 3e11 and _scratch(c) <= 5e9:
            return c


def _scratch(c):
    """Bytes of the largest tensor the plain form makes."""
    if c["op"] == "verify":
        return 4.0 * c["requests"] * (c["hi"] + c["drafts_hi"]) * max(LATENT + c["rope"], c["heads"] * c["drafts_hi"])
    return 0.0


def _draw(rng):
    op = rng.choice(["rotate", "rotate", "append", "append", "verify", "verify", "verify", "verify", "commit"])
    shape = rng.randrange(1 << 20)
    far = rng.choice([4095, 131071, 1048575])
    pairing = rng.choice(["adjacent", "halves"])
    source = rng.choice(["bf16", "fp32"])
    if op == "rotate":
        dim = rng.choice([64, 64, 128, 128, 192, 256, 512, 576, 8 * rng.randint(8, 72)])
        return dict(op=op, rows=_log_int(rng, 1, 16384), q_heads=rng.choice([1, 5, 8, 16, 32, 64, 100, 128]), k_heads=rng.choice([0, 1, 1, 3, 8]), dim=dim,
                    rope=rng.choice([r for r in (16, 32, 64, 64, 128) if r <= dim]), pairing=pairing, source=source, far=far, shape=shape)
    if op == "append":
        return dict(op=op, rows=_log_int(rng, 1, 65536), rope=rng.choice([0, 64, 64]), fmt=rng.choice([BF16, MXFP4]), source=source, pairing=pairing, far=far,
                    back=True, shape=shape)
    if op == "verify":
        hi = _log_int(rng, 1, 131072 if rng.random() < 0.3 else 32768)
        most = _log_int(rng, 1, 64)
        return dict(op=op, requests=_log_int(rng, 1, 48), lo=hi // 3 if rng.random() < 0.8 else 0, hi=hi, drafts_lo=max(1, most // 3), drafts_hi=most,
                    heads=rng.choice([1, 5, 8, 16, 16, 32, 64, 100, 128]), rope=rng.choice([0, 64, 64]), fmt=rng.choice([BF16, BF16, MXFP4]),
                    tree=rng.random() < 0.7, shape=shape)
    most = _log_int(rng, 1, 64)
    return dict(op=op, requests=_log_int(rng, 1, 64), layers=_log_int(rng, 1, 24), drafts_lo=max(1, most // 3), drafts_hi=most, rope=rng.choice([0, 64]),
                fmt=rng.choice([BF16, MXFP4]), shape=shape)


def _lengths(case, lo, hi, n, salt):
    """n lengths in [lo, hi], fixed by the case; the largest is among them."""
    r = random.Random("%s %s %s %s %s" % (case.get("shape", 7), lo, hi, n, salt))
    v = [r.randint(lo, hi) for _ in range(n)]
    v[r.randrange(n)] = hi
    return v


def _seen(case, drafts):
    """Of each request, the drafts that each draft sees, itself among them: a random tree (a parent is drafted before its
    children), or the chain."""
    r = random.Random("%s tree" % case.get("shape", 7))
    trees = []
    for n in drafts:
        seen = []
        for j in range(n):
            parent = (r.randint(max(-1, j - 8), j - 1) if r.random() < 0.6 else j - 1) if case["tree"] else j - 1
            seen.append((seen[parent] if parent >= 0 else 0) | 1 << j)
        trees.append(seen)
    return trees


def _paths(case, drafts):
    """Accepted drafts of each request, ascending: a start of the first ones, then drafts behind the accepted number, so that
    moving them twice is moving them once."""
    r = random.Random("%s path" % case.get("shape", 7))
    paths = []
    for n in drafts:
        take = r.randint(0, max(1, n // 2))
        same = r.randint(0, take)
        paths.append(list(range(same)) + sorted(r.sample(range(take, n), min(take - same, n - take))))
    return paths


def _record(fmt, rope):
    return 2 * (LATENT + rope) if fmt == BF16 else LATENT // 2 + LATENT // 32 + 2 * rope


def _pages(n):
    return (n + PAGE - 1) // PAGE


def _verify_sizes(case):
    base = _lengths(case, case["lo"], case["hi"], case["requests"], "len")
    return base, _lengths(case, case["drafts_lo"], case["drafts_hi"], case["requests"], "drafts")


def work(case):
    op = case["op"]
    if op == "rotate":
        n = case["rows"] * (case["q_heads"] + case["k_heads"]) * case["dim"]
        return {"bytes": n * ((4 if case["source"] == "fp32" else 2) + 2) + 4 * case["rows"], "flops": 0}
    if op == "append":
        row = (4 if case["source"] == "fp32" else 2) * (LATENT + case["rope"])
        rec = _record(case["fmt"], case["rope"])
        back = rec + 2 * (LATENT + case["rope"]) if case["back"] else 0
        return {"bytes": case["rows"] * (row + 12 + rec + back), "flops": 0}
    if op == "verify":
        base, drafts = _verify_sizes(case)
        pairs = sum(n * b for n, b in zip(drafts, base)) + sum(bin(m).count("1") for seen in _seen(case, drafts) for m in seen)
        rows = sum(drafts) * case["heads"]
        io = rows * (2 * (LATENT + case["rope"]) + 2 * LATENT + 4) + 8 * sum(drafts)
        return {"bytes": (sum(base) + sum(drafts)) * _record(case["fmt"], case["rope"]) + io, "flops": 2.0 * case["heads"] * (2 * LATENT + case["rope"]) * pairs}
    drafts = _lengths(case, case["drafts_lo"], case["drafts_hi"], case["requests"], "drafts")
    moved = sum(1 for path in _paths(case, drafts) for k, d in enumerate(path) if k != d)
    return {"bytes": 2 * moved * case["layers"] * _record(case["fmt"], case["rope"]) + 20 * case["requests"], "flops": 0}


# ------------------------------------------------------------------ inputs

def _table(lens, gen, dev, spare=3):
    """A shuffled page table for histories of `lens` records: (table [n, most], pages in the pool)."""
    counts = torch.tensor([_pages(n) for n in lens], device=dev)
    most, total = max(1, int(max(_pages(n) for n in lens))), int(sum(_pages(n) for n in lens))
    order = torch.randperm(total + spare, generator=gen, device=dev)[:total].int()
    table = torch.full((len(lens), most), -1, dtype=torch.int32, device=dev)
    at = torch.arange(most, device=dev)[None, :] < counts[:, None]
    table[at] = order
    return table, total + spare


def _pool(pages, fmt, rope, gen, dev):
    """A pool of pages full of records: N(0, 1) latents in bf16, or e2m1 codes with block scales 2^-3 .. 2^0."""
    if fmt == BF16:
        x = torch.randn(pages, PAGE, LATENT + rope, generator=gen, device=dev, dtype=torch.bfloat16)
        return x.view(torch.uint8).reshape(pages, -1)
    codes = torch.randint(0, 256, (pages, PAGE, LATENT // 2), generator=gen, device=dev, dtype=torch.uint8)
    scales = torch.randint(124, 128, (pages, PAGE, LATENT // 32), generator=gen, device=dev, dtype=torch.uint8)
    rest = torch.randn(pages, PAGE, rope, generator=gen, device=dev, dtype=torch.bfloat16).view(torch.uint8)
    return torch.cat([codes, scales, rest], 2).reshape(pages, -1).contiguous()


def _freq(rope, dev):
    """The usual frequencies 10000^(-2 j / rope), in the precision that a program keeps them."""
    return (10000.0 ** (-torch.arange(0, rope, 2, device=dev, dtype=torch.float64) / max(rope, 1))).float()


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev).manual_seed(seed)
    s = dict(case)
    op = case["op"]

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device=dev)

    def rows(n, width):
        """Rows of a projection's product, of sizes that differ from row to row."""
        x = torch.randn(n, width, generator=gen, device=dev, dtype=torch.float32)
        x *= torch.exp2(torch.randint(-3, 4, (n, 1), generator=gen, device=dev).float())
        return x.to(DTYPE[case["source"]])

    def weight(n):
        return 1.0 + 0.1 * torch.randn(n, generator=gen, device=dev, dtype=torch.float32)

    if op in ("rotate", "append"):
        n, rope = case["rows"], case["rope"]
        # positions of packed requests: runs that begin anywhere
        first = torch.randint(0, max(1, case["far"] - 4096), (n,), generator=gen, device=dev)
        s.update(pos=(first[torch.arange(n, device=dev) // 256 * 256] + torch.arange(n, device=dev) % 256).int(), freq=_freq(rope, dev))
    if op == "rotate":
        dim, qh, kh = case["dim"], case["q_heads"], case["k_heads"]
        x = rows(n, (qh + kh) * dim).view(n, qh + kh, dim)
        s.update(q=x[:, :qh], k=x[:, qh:] if kh else None, q_weight=weight(dim), k_weight=weight(dim) if kh else None)
    elif op == "append":
        table, pages = _table([n], gen, dev)
        at = torch.arange(n, device=dev)
        wide = LATENT + rope + 64  # the latents are the first columns of a wider product
        s.update(x=rows(n, wide)[:, :LATENT + rope], weight=weight(LATENT), slots=table[0].long()[at // PAGE] * PAGE + at % PAGE, page_table=table,
                 kv_start=ints([0, n]), pool=torch.zeros(pages, PAGE * _record(case["fmt"], rope), dtype=torch.uint8, device=dev), n_rows=n)
    elif op == "verify":
        base, drafts = _verify_sizes(case)
        table, pages = _table([b + n for b, n in zip(base, drafts)], gen, dev)
        start = [sum(drafts[:k]) for k in range(len(drafts) + 1)]
        bits = [m - (1 << 64) if m >> 63 else m for seen in _seen(case, drafts) for m in seen]
        s.update(pool=_pool(pages, case["fmt"], case["rope"], gen, dev), page_table=table, base_len=ints(base), row_start=ints(start),
                 mask=torch.tensor(bits, dtype=torch.int64, device=dev)[:, None] if case["tree"] else None, most=max(b + n for b, n in zip(base, drafts)),
                 most_drafts=max(drafts), q=torch.randn(start[-1], case["heads"], LATENT + case["rope"], generator=gen, device=dev, dtype=torch.bfloat16),
                 scale=192 ** -0.5)
    elif op == "commit":
        drafts = _lengths(case, case["drafts_lo"], case["drafts_hi"], case["requests"], "drafts")
        base = _lengths(case, 1, 2 * PAGE, case["requests"], "base")
        paths = _paths(case, drafts)
        wide = max(1, max(len(p) for p in paths))
        table, pages = _table([b + n for b, n in zip(base, drafts)], gen, dev)
        pool = torch.randint(0, 256, (case["layers"], pages, PAGE * _record(case["fmt"], case["rope"])), generator=gen, device=dev, dtype=torch.uint8)
        s.update(pool=pool, page_table=table, base_len=ints(base), draft_len=ints(drafts), path=ints([p + [-1] * (wide - len(p)) for p in paths]),
                 path_len=ints([len(p) for p in paths]), room=sum(_pages(b + n) - _pages(b) for b, n in zip(base, drafts)) + len(base))
    return s


# ------------------------------------------------------------------ plain forms

_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _values(records, fmt, rope):
    """Records [..., bytes] as the values they stand for, [..., 512 + rope], in fp32."""
    if fmt == BF16:
        return records.view(torch.bfloat16).float()
    codes, scales, rest = records[..., :LATENT // 2], records[..., LATENT // 2:LATENT // 2 + LATENT // 32], records[..., LATENT // 2 + LATENT // 32:]
    grid = torch.tensor(_E2M1 + tuple(-v for v in _E2M1), device=records.device)
    pair = torch.stack([codes & 15, codes >> 4], -1).long()
    v = grid[pair].reshape(*records.shape[:-1], LATENT // 32, 32) * torch.exp2(scales.float() - 127)[..., None]
    v = v.reshape(*records.shape[:-1], LATENT)
    return torch.cat([v, rest.contiguous().view(torch.bfloat16).float()], -1) if rope else v


def _norm(x, weight):
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * weight


def _turn(x, pos, freq, pairing):
    """x [rows, ..., rope] turned by pos * freq; the angles in 64 bits."""
    if x.shape[-1] == 0:
        return x
    t = pos.double()[:, None] * freq.double()[None, :]
    c, s = torch.cos(t).to(x.dtype), torch.sin(t).to(x.dtype)
    for _ in range(x.dim() - 2):
        c, s = c.unsqueeze(1), s.unsqueeze(1)
    if pairing == "adjacent":
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)
    a, b = x.chunk(2, -1)
    return torch.cat([a * c - b * s, b * c + a * s], -1)


def _plain_rotate(s):
    out = {}
    for name in ("q", "k"):
        if s[name] is None:
            continue
        y, still = _norm(s[name].float(), s[name + "_weight"]), s["dim"] - s["rope"]
        out[name] = torch.cat([y[..., :still], _turn(y[..., still:], s["pos"], s["freq"], s["pairing"])], -1).to(torch.bfloat16)
    return out


def _quantise(x):
    """MXFP4 records' codes and scale bytes of rows [n, 512]."""
    b = x.reshape(x.shape[0], LATENT // 32, 32)
    amax = b.abs().amax(-1)
    e = torch.where(amax > 0, torch.frexp(amax)[1] - 3, torch.full_like(amax, -127).int()).clamp(-127, 127)
    y = (b * torch.exp2(-e.to(x.dtype))[..., None]).abs()
    m = (y > 0.25).int() + (y >= 0.75) + (y > 1.25) + (y >= 1.75) + (y > 2.5) + (y >= 3.5) + (y > 5.0)
    code = (m | (torch.signbit(b).int() << 3)).to(torch.uint8).reshape(x.shape[0], LATENT // 2, 2)
    return code[..., 0] | (code[..., 1] << 4), (e + 127).to(torch.uint8)


def _plain_append(s):
    rope, pool = s["rope"], s["pool"]
    turned = _turn(s["x"][:, LATENT:].float(), s["pos"], s["freq"], s["pairing"]).to(torch.bfloat16).contiguous().view(torch.uint8)
    if s["fmt"] == BF16:
        rec = torch.cat([_norm(s["x"][:, :LATENT].float(), s["weight"]).to(torch.bfloat16).view(torch.uint8), turned], 1)
    else:  # in 64 bits: values lie next to the borders between two codes
        codes, scales = _quantise(_norm(s["x"][:, :LATENT].double(), s["weight"].double()))
        rec = torch.cat([codes, scales, turned], 1)
    pool.view(-1, rec.shape[1])[s["slots"]] = rec
    return _plain_read(s) if s["back"] else pool.view(torch.bfloat16)


def _plain_read(s):
    start, table = s["kv_start"].long(), s["page_table"].long()
    i = torch.arange(s["n_rows"], device=start.device)
    req = torch.searchsorted(start[1:], i, right=True)
    pos = i - start[req]
    rec = s["pool"].view(-1, _record(s["fmt"], s["rope"]))[table[req, pos // PAGE] * PAGE + pos % PAGE]
    return _values(rec, s["fmt"], s["rope"]).to(torch.bfloat16)


def _plain_verify(s):
    """All requests padded to the longest, all of their drafts at once."""
    records, table, base, start = s["pool"].view(-1, _record(s["fmt"], s["rope"])), s["page_table"].long(), s["base_len"].long(), s["row_start"].long()
    dev, n, h, most = base.device, start[1:] - start[:-1], s["heads"], s["most_drafts"]
    pos = torch.arange(s["most"], device=dev)
    at = table[:, pos // PAGE].clamp(min=0) * PAGE + pos % PAGE
    k = _values(records[torch.where(pos[None, :] < (base + n)[:, None], at, at[:, :1])], s["fmt"], s["rope"])
    j = torch.arange(most, device=dev)
    there = j[None, :] < n[:, None]
    row = torch.where(there, start[:-1, None] + j[None, :], torch.zeros_like(there).long())
    draft = pos[None, :] - base[:, None]  # [requests, most]
    if s["mask"] is None:
        sees = draft[:, None, :] <= j[None, :, None]
    else:
        bits = s["mask"][row, 0]
        sees = (draft < 0)[:, None, :] | ((bits[:, :, None] >> draft.clamp(0, 63)[:, None, :]) & 1 > 0)
    sees = sees & (draft < n[:, None])[:, None, :]
    z = torch.matmul(s["q"][row].float().flatten(1, 2), k.transpose(1, 2)) * s["scale"]
    z = z.view(len(n), most, h, -1).masked_fill(~sees[:, :, None, :], -math.inf)
    top = z.amax(-1, keepdim=True)
    z = torch.exp(z - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = z.sum(-1, keepdim=True)
    o = torch.matmul(z.flatten(1, 2), k[..., :LATENT]).view(len(n), most, h, LATENT) / total.clamp(min=1e-30)
    return {"out": o[there].to(torch.bfloat16), "lse": (torch.log(total) + top).squeeze(-1)[there]}


def _plain_commit(s):
    pool, table, base, path, took = s["pool"], s["page_table"].long(), s["base_len"].long(), s["path"].long(), s["path_len"].long()
    layers, k = pool.shape[0], torch.arange(path.shape[1], device=base.device)
    live = k[None, :] < took[:, None]
    req = torch.arange(base.numel(), device=base.device)[:, None].expand_as(live)[live]

    def slot(pos):
        return table[req, pos // PAGE] * PAGE + pos % PAGE

    records = pool.view(layers, -1, _record(s["fmt"], s["rope"]))
    records[:, slot((base[:, None] + k[None, :])[live])] = records[:, slot((base[:, None] + path)[live])]
    new_len = base + took
    p = torch.arange(table.shape[1], device=base.device)[None, :]
    back = (p >= ((new_len + PAGE - 1) // PAGE)[:, None]) & (p < ((base + s["draft_len"] + PAGE - 1) // PAGE)[:, None])
    rank = torch.cumsum(back.flatten(), 0) - 1
    free = torch.full((s["room"] + 1,), -1, dtype=torch.int32, device=base.device)
    free[torch.where(back.flatten(), rank, s["room"])] = s["page_table"].flatten()
    free[s["room"]] = -1
    return {"pool": _stand_for(pool, s), "new_len": new_len.int(), "freed": free[:-1], "n_freed": (rank[-1:] + 1).int()}


def _stand_for(pool, s):
    """The cache of every layer, as 16-bit words: records move whole, whatever they hold."""
    return pool.view(torch.int16)


# ------------------------------------------------------------------ one pass

def run(state):
    s = state
    op = s["op"]
    if not own:
        return {"rotate": _plain_rotate, "append": _plain_append, "verify": _plain_verify, "commit": _plain_commit}[op](s)
    from sparse_attention_kv_e4m3_gb300 import draft, latent

    if op == "rotate":
        q, k = draft.csa_head_norm_rotate(s["q"], s["pos"], s["freq"], k=s["k"], q_weight=s["q_weight"], k_weight=s["k_weight"], eps=EPS, pairing=s["pairing"])
        return {"q": q} if k is None else {"q": q, "k": k}
    cache = s.get("cache")
    if cache is None:  # the handle that a program keeps beside its pages
        kind = draft.LayeredCache if op == "commit" else latent.LatentCache
        cache = s["cache"] = kind(s["pool"], rope_dim=s["rope"], record_format=s["fmt"])
    if op == "append":
        draft.csa_latent_append(s["x"], s["slots"], s["pos"], cache, s["freq"], weight=s["weight"], eps=EPS, pairing=s["pairing"])
        return latent.csa_latent_read(cache, s["page_table"], s["kv_start"], s["n_rows"]) if s["back"] else s["pool"].view(torch.bfloat16)
    if op == "verify":
        out, lse = draft.csa_draft_attend(s["q"], cache, s["page_table"], s["base_len"], s["row_start"], scale=s["scale"], mask=s["mask"])
        return {"out": out, "lse": lse}
    done = draft.csa_draft_commit(cache, s["page_table"], s["base_len"], s["draft_len"], s["path"], s["path_len"], room=s["room"])
    return {"pool": _stand_for(s["pool"], s), "new_len": done.new_len, "freed": done.freed, "n_freed": done.n_freed}


# ------------------------------------------------------------------ the definition in 64 bits

def _exact_values(rows, fmt, rope):
    """Records [n, bytes] in 64 bits, the 4-bit values by the format's formula."""
    if fmt == BF16:
        return rows.contiguous().view(torch.bfloat16).double()
    nibbles = torch.stack([rows[:, :LATENT // 2] & 15, rows[:, :LATENT // 2] >> 4], 2).reshape(-1, LATENT).long()
    sign, e, m = 1.0 - 2.0 * (nibbles >> 3).double(), ((nibbles >> 1) & 3).double(), (nibbles & 1).double()
    v = sign * torch.where(e > 0, (1 + 0.5 * m) * 2.0 ** (e - 1), 0.5 * m)
    v = v * (2.0 ** (rows[:, LATENT // 2:LATENT // 2 + LATENT // 32].double() - 127)).repeat_interleave(32, 1)
    return torch.cat([v, rows[:, LATENT // 2 + LATENT // 32:].contiguous().view(torch.bfloat16).double()], 1) if rope else v


def _exact_turn(x, pos, freq, pairing):
    """x [rows, heads, rope] in 64 bits, as complex numbers times e^(i pos freq)."""
    if x.shape[-1] == 0:
        return x
    angle = torch.outer(pos.double(), freq.double())
    turn = torch.polar(torch.ones_like(angle), angle)[:, None, :]
    if pairing == "adjacent":
        return torch.view_as_real(torch.view_as_complex(x.reshape(*x.shape[:-1], -1, 2).contiguous()) * turn).flatten(-2)
    half = x.shape[-1] // 2
    y = torch.complex(x[..., :half].contiguous(), x[..., half:].contiguous()) * turn
    return torch.cat([y.real, y.imag], -1)


def _exact_norm(x, weight):
    return weight.double() * x / ((x ** 2).sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt()


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "rotate":
        out = {}
        for name in ("q", "k"):
            if s[name] is not None:
                y = _exact_norm(s[name].double(), s[name + "_weight"])
                cut = case["dim"] - case["rope"]
                y[..., cut:] = _exact_turn(y[..., cut:].clone(), s["pos"], s["freq"], case["pairing"])
                out[name] = y
        return out
    if op == "append":
        rope, fmt = case["rope"], case["fmt"]
        x = s["x"].double()
        turned = _exact_turn(x[:, None, LATENT:], s["pos"], s["freq"], case["pairing"])[:, 0]
        y = _exact_norm(x[:, :LATENT], s["weight"])
        if fmt == MXFP4:
            b = y.reshape(-1, 32)
            unit = torch.ldexp(torch.ones_like(b[:, :1]), torch.frexp(b.abs().amax(1, keepdim=True))[1] - 3)
            y = b / unit
            # the spacing of e2m1 at each magnitude: 1/2 below 2, 1 below 4, 2 above; round() takes ties to even
            step = torch.where(y.abs() < 2, 0.5, torch.where(y.abs() < 4, 1.0, 2.0))
            y = ((torch.round(y / step) * step).clamp(-6, 6) * unit).reshape(-1, LATENT)
        y = torch.cat([y, turned], 1)
        if case["back"]:
            return y
        pool = s["pool"].view(torch.bfloat16).double().reshape(-1, LATENT + rope)
        pool[s["slots"]] = y
        return pool.reshape(s["pool"].shape[0], -1)
    if op == "verify":
        base, drafts = _verify_sizes(case)
        records, outs, lses, at_row = s["pool"].view(-1, _record(case["fmt"], case["rope"])), [], [], 0
        for r, (b, n, seen) in enumerate(zip(base, drafts, _seen(case, drafts))):
            pages = s["page_table"][r, :_pages(b + n)].long()
            k = _exact_values(records.view(s["pool"].shape[0], PAGE, -1)[pages].flatten(0, 1)[:b + n], case["fmt"], case["rope"])
            hidden = torch.tensor([[not seen[j] >> i & 1 for i in range(n)] for j in range(n)], device=k.device)
            for j in range(n):
                z = (s["q"][at_row + j].double() @ k.t()) * s["scale"]
                z[:, b:] = z[:, b:].masked_fill(hidden[j], -math.inf)
                lses.append(torch.logsumexp(z, 1))
                outs.append(torch.softmax(z, 1) @ k[:, :LATENT])
            at_row += n
        return {"out": torch.stack(outs), "lse": torch.stack(lses)}
    # whole numbers: a record at a time, on the host
    drafts = _lengths(case, case["drafts_lo"], case["drafts_hi"], case["requests"], "drafts")
    pool, table = s["pool"].cpu(), s["page_table"].tolist()
    rec = _record(case["fmt"], case["rope"])
    new_len, freed = [], []
    for r, (b, n, path) in enumerate(zip(s["base_len"].tolist(), drafts, _paths(case, drafts))):
        for k, d in enumerate(path):
            to, of = b + k, b + d
            chunk = pool[:, table[r][of // PAGE], of % PAGE * rec:(of % PAGE + 1) * rec].clone()
            pool[:, table[r][to // PAGE], to % PAGE * rec:(to % PAGE + 1) * rec] = chunk
        new_len.append(b + len(path))
        freed += table[r][_pages(b + len(path)):_pages(b + n)]
    return {"pool": pool.view(torch.int16), "new_len": torch.tensor(new_len, dtype=torch.int32),
            "freed": torch.tensor(freed + [-1] * (s["room"] - len(freed)), dtype=torch.int32), "n_freed": torch.tensor([len(freed)], dtype=torch.int32)}
