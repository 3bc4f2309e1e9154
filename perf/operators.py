"""Measured cases of the latent-cache operators: block tables, the latent cache's writer and reader, and
latent attention in its absorbed form (over a paged cache) and its expanded form (over prompts).

`run` computes an operator in elementary torch operations, or, where `own` is set, calls the library.
"""
import math
import random

import torch

own = False

PAGE = 64          # records a page
LATENT = 512       # latent values of a record: keys and values
NOPE, ROPE, VDIM = 128, 64, 128   # expanded head: key values without and with rope, values
BF16, MXFP4 = "bf16", "mxfp4"


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one decode step of the long ragged batch: 64 requests, one new record each
        dict(name="tables_decode", op="tables", requests=64, old_lo=65536, old_hi=131071, new_lo=1, new_hi=1),
        # admission of a large wave of ragged prompts, some requests idle
        dict(name="tables_prompts", op="tables", requests=509, old_lo=0, old_hi=8192, new_lo=0, new_hi=4096),
        # the records of one decode step stored in the bf16 cache
        dict(name="store_decode_bf16", op="store", rows=64, rope=64, fmt=BF16, source="bf16", back=False),
        # the latents of a wave of prompts, fp32 out of the norm, stored in 4 bits and read back for expansion
        dict(name="store_read_mxfp4", op="store", rows=65537, rope=64, fmt=MXFP4, source="fp32", back=True),
        # a request's history of the chunked prefill read back out of its shuffled pages
        dict(name="read_history_bf16", op="read", requests=3, lo=5001, hi=16384, rope=64, fmt=BF16),
        # one row of a small request, few heads of a sharded layer: latency
        dict(name="attend_one_row", op="attend", rows=1, heads=16, rope=64, fmt=BF16, mode="all", lo=1000, hi=1000, top=0, shared=False),
        # the consumer of the indexer: 64 decode rows, their top 512 positions out of long histories
        dict(name="attend_top512_decode", op="attend", rows=64, heads=64, rope=64, fmt=BF16, mode="top", lo=16384, hi=32768, top=512, shared=False),
        # few very long histories read whole
        dict(name="attend_long_rows", op="attend", rows=4, heads=64, rope=0, fmt=BF16, mode="all", lo=65536, hi=131072, top=0, shared=False),
        # the decode batch over a cache held in 4 bits
        dict(name="attend_4bit_batch", op="attend", rows=32, heads=64, rope=64, fmt=MXFP4, mode="all", lo=30001, hi=32768, top=0, shared=False),
        # a prompt chunk of one request, every row with its own 512 positions, all heads on one GPU
        dict(name="attend_top512_chunk", op="attend", rows=1024, heads=128, rope=64, fmt=BF16, mode="top", lo=16384, hi=16384, top=512, shared=True),
        # a wave of ragged prompts
        dict(name="prefill_ragged", op="prefill", requests=8, heads=32, new_lo=130, new_hi=2048, old_lo=0, old_hi=0),
        # a chunk of 4096 new tokens against a history
        dict(name="prefill_chunk", op="prefill", requests=1, heads=16, new_lo=4096, new_hi=4096, old_lo=12288, old_hi=12288),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    while True:
        c = _draw(rng)
        w = work(c)
        if w["bytes"] <= 6e8 and w["flops"] <= 2.5e11 and _scratch(c) <= 6e9:
            return c


def _scratch(c):
    """Bytes of the largest tensor the plain form makes."""
    if c["op"] == "attend":
        span = c["top"] if c["mode"] == "top" else c["hi"]
        return 4.0 * c["rows"] * span * max(LATENT + c["rope"], c["heads"])
    if c["op"] == "prefill":
        return 4.0 * c["requests"] * c["heads"] * c["new_hi"] * (c["new_hi"] + c["old_hi"])
    return 0.0


def _draw(rng):
    op = rng.choice(["tables", "store", "read", "attend", "attend", "attend", "prefill", "prefill"])
    shape = rng.randrange(1 << 20)
    if op == "tables":
        if rng.random() < 0.5:
            hi = _log_int(rng, 64, 131071)
            return dict(op=op, requests=_log_int(rng, 1, 1024), old_lo=0, old_hi=hi, new_lo=0, new_hi=rng.randint(1, 4), shape=shape)
        return dict(op=op, requests=_log_int(rng, 1, 512), old_lo=0, old_hi=_log_int(rng, 1, 8192), new_lo=0, new_hi=_log_int(rng, 1, 4096), shape=shape)
    if op == "store":
        return dict(op=op, rows=_log_int(rng, 1, 65536), rope=rng.choice([0, 64]), fmt=rng.choice([BF16, MXFP4]),
                    source=rng.choice(["bf16", "fp32"]), back=True, shape=shape)
    if op == "read":
        hi = _log_int(rng, 1, 16384)
        return dict(op=op, requests=_log_int(rng, 1, 16), lo=max(1, hi // 3), hi=hi, rope=rng.choice([0, 64]), fmt=rng.choice([BF16, MXFP4]), shape=shape)
    if op == "attend":
        top = rng.random() < 0.5
        shared = top and rng.random() < 0.3
        hi = _log_int(rng, 1, 32768 if top or rng.random() < 0.7 else 131072)
        return dict(op=op, rows=_log_int(rng, 1, 1024 if shared else 64), heads=rng.choice([1, 5, 8, 16, 32, 64, 64, 100, 128]), rope=rng.choice([0, 64]),
                    fmt=rng.choice([BF16, MXFP4]), mode="top" if top else "all", lo=max(1, hi // 2), hi=hi,
                    top=rng.choice([512, 512, rng.randint(1, 1024)]) if top else 0, shared=shared, shape=shape)
    new = _log_int(rng, 1, 4096)
    old = 0 if rng.random() < 0.5 else _log_int(rng, 1, 12288)
    return dict(op=op, requests=_log_int(rng, 1, 16), heads=rng.choice([1, 3, 8, 16, 32, 64]), new_lo=max(1, new // 4), new_hi=new, old_lo=old // 3, old_hi=old, shape=shape)


def _lengths(case, lo, hi, n, salt):
    """n lengths in [lo, hi], fixed by the case; the largest is among them."""
    r = random.Random("%s %s %s %s %s" % (case.get("shape", 7), lo, hi, n, salt))
    v = [r.randint(lo, hi) for _ in range(n)]
    v[r.randrange(n)] = hi
    return v


def _record(fmt, rope):
    return 2 * (LATENT + rope) if fmt == BF16 else LATENT // 2 + LATENT // 32 + 2 * rope


def _pages(n):
    return (n + PAGE - 1) // PAGE


def work(case):
    op = case["op"]
    if op == "tables":
        old = _lengths(case, case["old_lo"], case["old_hi"], case["requests"], "old")
        new = _lengths(case, case["new_lo"], case["new_hi"], case["requests"], "new")
        fresh = sum(_pages(a + b) - _pages(a) for a, b in zip(old, new))
        return {"bytes": 8 * len(old) + 12 * len(old) + 8 * fresh + 20 * sum(new), "flops": 0}
    if op == "store":
        row = (4 if case["source"] == "fp32" else 2) * (LATENT + case["rope"])
        rec = _record(case["fmt"], case["rope"])
        back = rec + 2 * (LATENT + case["rope"]) if case["back"] else 0
        return {"bytes": case["rows"] * (row + 8 + rec + back), "flops": 0}
    if op == "read":
        n = sum(_lengths(case, case["lo"], case["hi"], case["requests"], "len"))
        return {"bytes": n * (_record(case["fmt"], case["rope"]) + 2 * (LATENT + case["rope"])), "flops": 0}
    if op == "attend":
        lens = _lengths(case, case["lo"], case["hi"], case["rows"], "len")
        seen = [min(n, case["top"]) for n in lens] if case["mode"] == "top" else lens
        rec = _record(case["fmt"], case["rope"])
        distinct = min(sum(seen), case["hi"]) if case["shared"] else sum(seen)
        io = case["rows"] * case["heads"] * (2 * (LATENT + case["rope"]) + 2 * LATENT + 4)
        return {"bytes": distinct * rec + io + (4 * case["rows"] * case["top"]), "flops": 2.0 * case["heads"] * (2 * LATENT + case["rope"]) * sum(seen)}
    new = _lengths(case, case["new_lo"], case["new_hi"], case["requests"], "new")
    old = _lengths(case, case["old_lo"], case["old_hi"], case["requests"], "old")
    pairs = sum(n * o + n * (n + 1) // 2 for n, o in zip(new, old))
    tq, tk, h = sum(new), sum(new) + sum(old), case["heads"]
    return {"bytes": 2 * tq * h * (NOPE + ROPE + VDIM) + 4 * tq * h + 2 * tk * (h * (NOPE + VDIM) + ROPE), "flops": 2.0 * h * (NOPE + ROPE + VDIM) * pairs}


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


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev).manual_seed(seed)
    s = dict(case)
    op = case["op"]

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device=dev)

    if op == "tables":
        old = _lengths(case, case["old_lo"], case["old_hi"], case["requests"], "old")
        new = _lengths(case, case["new_lo"], case["new_hi"], case["requests"], "new")
        # the page table as the last step left it, the pool's free pages in the order they are handed out
        table, held = _table(old, gen, dev, spare=0)
        width = max(_pages(a + b) for a, b in zip(old, new)) + 1
        wide = torch.full((len(old), width), -1, dtype=torch.int32, device=dev)
        wide[:, :min(width, table.shape[1])] = table[:, :width]
        fresh = sum(_pages(a + b) - _pages(a) for a, b in zip(old, new))
        free = (held + torch.randperm(fresh + 5, generator=gen, device=dev)).int()
        s.update(old_len=ints(old), new_len=ints(new), page_table=wide, free_pages=free, n_rows=sum(new) + 3)
    elif op == "store":
        n, rope = case["rows"], case["rope"]
        table, pages = _table([n], gen, dev)
        dtype = torch.bfloat16 if case["source"] == "bf16" else torch.float32
        x = torch.randn(n, LATENT + rope, generator=gen, device=dev, dtype=torch.float32)
        x *= torch.exp2(torch.randint(-3, 4, (n, 1), generator=gen, device=dev).float())
        at = torch.arange(n, device=dev)
        slots = table[0].long()[at // PAGE] * PAGE + at % PAGE
        pool = torch.zeros(pages, PAGE * _record(case["fmt"], rope), dtype=torch.uint8, device=dev)
        s.update(x=x.to(dtype), slots=slots, page_table=table, kv_start=ints([0, n]), pool=pool, n_rows=n)
    elif op == "read":
        lens = _lengths(case, case["lo"], case["hi"], case["requests"], "len")
        table, pages = _table(lens, gen, dev)
        start = [sum(lens[:k]) for k in range(len(lens) + 1)]
        s.update(pool=_pool(pages, case["fmt"], case["rope"], gen, dev), page_table=table, kv_start=ints(start), n_rows=start[-1])
    elif op == "attend":
        lens = _lengths(case, case["lo"], case["hi"], case["rows"], "len")
        table, pages = _table([case["hi"]] if case["shared"] else lens, gen, dev)
        if case["shared"]:
            lens = [min(n, case["hi"]) for n in lens]
        wide = LATENT + case["rope"]
        s.update(pool=_pool(pages, case["fmt"], case["rope"], gen, dev), page_table=table, row_len=ints(lens), idx=None,
                 row_req=torch.zeros(case["rows"], dtype=torch.int32, device=dev) if case["shared"] else None,
                 q=torch.randn(case["rows"], case["heads"], wide, generator=gen, device=dev, dtype=torch.bfloat16), scale=(NOPE + ROPE) ** -0.5)
        if case["mode"] == "top":
            # distinct positions in the order the indexer ranks them, -1 past a short history
            top, n = case["top"], s["row_len"].long()
            if case["hi"] * case["rows"] <= 1 << 26:
                r = torch.rand(case["rows"], max(case["hi"], top), generator=gen, device=dev)
                r.masked_fill_(torch.arange(r.shape[1], device=dev)[None, :] >= n[:, None], -1.0)
                val, idx = torch.topk(r, top, dim=1)
                s["idx"] = torch.where(val >= 0, idx, torch.full_like(idx, -1)).int()
            else:
                raise ValueError("too many candidate positions")
    else:
        new = _lengths(case, case["new_lo"], case["new_hi"], case["requests"], "new")
        old = _lengths(case, case["old_lo"], case["old_hi"], case["requests"], "old")
        full = [a + b for a, b in zip(new, old)]
        tq, tk, h = sum(new), sum(full), case["heads"]
        kv = torch.randn(tk, h, NOPE + VDIM, generator=gen, device=dev, dtype=torch.bfloat16)  # one expansion product's result
        latent = torch.randn(tk, LATENT + ROPE, generator=gen, device=dev, dtype=torch.bfloat16)
        s.update(q=torch.randn(tq, h, NOPE + ROPE, generator=gen, device=dev, dtype=torch.bfloat16), k_nope=kv[..., :NOPE], v=kv[..., NOPE:],
                 k_rope=latent[:, LATENT:], q_start=ints([sum(new[:k]) for k in range(len(new) + 1)]),
                 kv_start=ints([sum(full[:k]) for k in range(len(full) + 1)]), scale=(NOPE + ROPE) ** -0.5, most_q=max(new), most_k=max(full))
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


def _plain_tables(s):
    old, new, table = s["old_len"].long(), s["new_len"].long(), s["page_table"]
    total = old + new
    first, last = (old + PAGE - 1) // PAGE, (total + PAGE - 1) // PAGE
    taken = torch.cumsum(last - first, 0)
    p = torch.arange(table.shape[1], device=table.device)[None, :]
    source = (taken - (last - first))[:, None] + p - first[:, None]
    fresh = (p >= first[:, None]) & (p < last[:, None])
    table.copy_(torch.where(fresh, s["free_pages"][source.clamp(0, s["free_pages"].numel() - 1)], table))
    zero = torch.zeros(1, dtype=torch.long, device=table.device)
    row_start, kv_start = torch.cat([zero, torch.cumsum(new, 0)]), torch.cat([zero, torch.cumsum(total, 0)])
    i = torch.arange(s["n_rows"], device=table.device)
    req = torch.searchsorted(row_start[1:], i, right=True)
    live = req < old.numel()
    req = torch.where(live, req, torch.zeros_like(req))
    pos = old[req] + i - row_start[req]
    page = table[req, (pos // PAGE).clamp(0, table.shape[1] - 1)].long()
    return {"page_table": table, "row_req": req.int(), "row_pos": torch.where(live, pos, -1).int(), "row_len": torch.where(live, pos + 1, 0).int(),
            "row_slot": torch.where(live, page * PAGE + pos % PAGE, -1), "row_start": row_start.int(), "kv_start": kv_start.int(), "taken": taken[-1:].int()}


def _quantise(x):
    """MXFP4 records' codes and scale bytes of fp32 rows [n, 512]."""
    b = x.reshape(x.shape[0], LATENT // 32, 32)
    amax = b.abs().amax(-1)
    e = torch.where(amax > 0, torch.frexp(amax)[1] - 3, torch.full_like(amax, -127).int()).clamp(-127, 127)
    y = (b * torch.exp2(-e.float())[..., None]).abs()
    m = (y > 0.25).int() + (y >= 0.75) + (y > 1.25) + (y >= 1.75) + (y > 2.5) + (y >= 3.5) + (y > 5.0)
    code = (m | (torch.signbit(b).int() << 3)).to(torch.uint8).reshape(x.shape[0], LATENT // 2, 2)
    return code[..., 0] | (code[..., 1] << 4), (e + 127).to(torch.uint8)


def _plain_store(s):
    x, rope, pool = s["x"].float(), s["rope"], s["pool"]
    if s["fmt"] == BF16:
        rec = x.to(torch.bfloat16).view(torch.uint8)
    else:
        codes, scales = _quantise(x[:, :LATENT])
        rec = torch.cat([codes, scales, x[:, LATENT:].to(torch.bfloat16).view(torch.uint8)], 1)
    pool.view(-1, rec.shape[1])[s["slots"]] = rec
    return _plain_read(s) if s["back"] else pool.view(torch.bfloat16)


def _plain_read(s):
    start, table = s["kv_start"].long(), s["page_table"].long()
    i = torch.arange(s["n_rows"], device=start.device)
    req = torch.searchsorted(start[1:], i, right=True)
    pos = i - start[req]
    rec = s["pool"].view(-1, _record(s["fmt"], s["rope"]))[table[req, pos // PAGE] * PAGE + pos % PAGE]
    return _values(rec, s["fmt"], s["rope"]).to(torch.bfloat16)


def _softmax_parts(z, live):
    """exp(z - max) over the last axis with dead entries 0, and the log of the sum: -inf where nothing is live."""
    z = z.masked_fill(~live, -math.inf)
    top = z.amax(-1, keepdim=True)
    p = torch.exp(z - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = p.sum(-1, keepdim=True)
    return p, total, (torch.log(total) + top).squeeze(-1)


def _plain_attend(s):
    rec, rope = _record(s["fmt"], s["rope"]), s["rope"]
    records, table, n = s["pool"].view(-1, rec), s["page_table"].long(), s["row_len"].long()
    rows = n.numel()
    req = s["row_req"].long() if s["row_req"] is not None else torch.arange(rows, device=n.device)
    pos = s["idx"].long() if s["idx"] is not None else torch.arange(s["hi"], device=n.device)[None, :].expand(rows, -1)
    live = (pos >= 0) & (pos < n[:, None])
    pos = torch.where(live, pos, torch.zeros_like(pos))
    k = _values(records[table[req[:, None], pos // PAGE].clamp(min=0) * PAGE + pos % PAGE], s["fmt"], rope)
    z = torch.matmul(s["q"].float(), k.transpose(1, 2)) * s["scale"]
    p, total, lse = _softmax_parts(z, live[:, None, :])
    o = torch.matmul(p, k[..., :LATENT]) / total.clamp(min=1e-30)
    return {"out": o.to(torch.bfloat16), "lse": lse}


def _padded(x, start, most):
    """Rows start[r] .. start[r + 1] of x as [requests, most, ...], and which of them are there."""
    at = start[:-1, None] + torch.arange(most, device=x.device)[None, :]
    live = at < start[1:, None]
    return x[torch.where(live, at, torch.zeros_like(at))], live


def _plain_prefill(s):
    qs, ks = s["q_start"].long(), s["kv_start"].long()
    q, live_q = _padded(s["q"], qs, s["most_q"])
    kn, live_k = _padded(s["k_nope"], ks, s["most_k"])
    kr, v = _padded(s["k_rope"], ks, s["most_k"])[0], _padded(s["v"], ks, s["most_k"])[0]
    h = q.shape[2]
    k = torch.cat([kn, kr[:, :, None, :].expand(-1, -1, h, -1)], 3).float().permute(0, 2, 3, 1)
    z = torch.matmul(q.float().permute(0, 2, 1, 3), k) * s["scale"]
    i, j = torch.arange(s["most_q"], device=z.device), torch.arange(s["most_k"], device=z.device)
    past = ((ks[1:] - ks[:-1]) - (qs[1:] - qs[:-1]))[:, None, None]
    live = (j[None, None, :] <= i[None, :, None] + past) & live_k[:, None, :]
    p, total, lse = _softmax_parts(z, live[:, None])
    o = (torch.matmul(p, v.float().permute(0, 2, 1, 3)) / total.clamp(min=1e-30)).permute(0, 2, 1, 3)
    flat = qs[:-1, None] + i[None, :]
    at = torch.where(live_q, flat, torch.full_like(flat, s["q"].shape[0]))  # rows that are not there go to a row of their own
    out = torch.zeros(s["q"].shape[0] + 1, h, VDIM, dtype=torch.bfloat16, device=z.device)
    out[at] = o.to(torch.bfloat16)
    ls = torch.zeros(s["q"].shape[0] + 1, h, dtype=torch.float32, device=z.device)
    ls[at] = lse.permute(0, 2, 1)
    return {"out": out[:-1], "lse": ls[:-1]}


# ------------------------------------------------------------------ one pass

def run(state):
    s = state
    op = s["op"]
    if not own:
        return {"tables": _plain_tables, "store": _plain_store, "read": _plain_read, "attend": _plain_attend, "prefill": _plain_prefill}[op](s)
    from sparse_attention_kv_e4m3_gb300 import latent

    if op == "tables":
        t = latent.csa_build_tables(s["old_len"], s["new_len"], s["page_table"], s["free_pages"], s["n_rows"])
        return {"page_table": s["page_table"], "row_req": t.row_req, "row_pos": t.row_pos, "row_len": t.row_len, "row_slot": t.row_slot,
                "row_start": t.row_start, "kv_start": t.kv_start, "taken": t.taken}
    if op == "prefill":
        out, lse = latent.csa_latent_prefill(s["q"], s["k_nope"], s["k_rope"], s["v"], s["q_start"], s["kv_start"], scale=s["scale"])
        return {"out": out, "lse": lse}
    cache = s.get("cache")
    if cache is None:  # the handle that a program keeps beside its pages
        cache = s["cache"] = latent.LatentCache(s["pool"], rope_dim=s["rope"], record_format=s["fmt"])
    if op == "store":
        latent.csa_latent_write(s["x"], s["slots"], cache)
        return latent.csa_latent_read(cache, s["page_table"], s["kv_start"], s["n_rows"]) if s["back"] else s["pool"].view(torch.bfloat16)
    if op == "read":
        return latent.csa_latent_read(cache, s["page_table"], s["kv_start"], s["n_rows"])
    out, lse = latent.csa_latent_attend(s["q"], cache, s["page_table"], s["row_len"], scale=s["scale"], idx=s["idx"], row_req=s["row_req"])
    return {"out": out, "lse": lse}


# ------------------------------------------------------------------ the definition in 64 bits

def _exact_values(rows, fmt, rope):
    """Records [n, bytes] in 64 bits, the 4-bit values by the format's formula."""
    if fmt == BF16:
        return rows.view(torch.bfloat16).double()
    nibbles = torch.stack([rows[:, :LATENT // 2] & 15, rows[:, :LATENT // 2] >> 4], 2).reshape(-1, LATENT).long()
    sign, e, m = 1.0 - 2.0 * (nibbles >> 3).double(), ((nibbles >> 1) & 3).double(), (nibbles & 1).double()
    v = sign * torch.where(e > 0, (1 + 0.5 * m) * 2.0 ** (e - 1), 0.5 * m)
    v = v * (2.0 ** (rows[:, LATENT // 2:LATENT // 2 + LATENT // 32].double() - 127)).repeat_interleave(32, 1)
    return torch.cat([v, rows[:, LATENT // 2 + LATENT // 32:].contiguous().view(torch.bfloat16).double()], 1) if rope else v


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "tables":
        old, new, table, free = s["old_len"].tolist(), s["new_len"].tolist(), s["page_table"].tolist(), s["free_pages"].tolist()
        req, pos, length, slot, row_start, kv_start, taken = [], [], [], [], [0], [0], 0
        for r, (a, b) in enumerate(zip(old, new)):
            take = _pages(a + b) - _pages(a)
            table[r][_pages(a):_pages(a) + take] = free[taken:taken + take]
            taken += take
            req += [r] * b
            pos += range(a, a + b)
            length += range(a + 1, a + b + 1)
            slot += [table[r][n // PAGE] * PAGE + n % PAGE for n in range(a, a + b)]
            row_start.append(row_start[-1] + b)
            kv_start.append(kv_start[-1] + a + b)
        blank = s["n_rows"] - len(req)

        def ints(v, dtype=torch.int32):
            return torch.tensor(v, dtype=dtype)

        return {"page_table": ints(table), "row_req": ints(req + [0] * blank), "row_pos": ints(pos + [-1] * blank), "row_len": ints(length + [0] * blank),
                "row_slot": ints(slot + [-1] * blank, torch.int64), "row_start": ints(row_start), "kv_start": ints(kv_start), "taken": ints([taken])}
    if op in ("store", "read"):
        rope, fmt = case["rope"], case["fmt"]
        if op == "read":
            table, rec = s["page_table"].long(), _record(fmt, rope)
            rows = torch.cat([s["pool"][table[r, :_pages(b - a)]].reshape(-1, rec)[:b - a]
                              for r, (a, b) in enumerate(zip(s["kv_start"].tolist(), s["kv_start"].tolist()[1:]))])
            return _exact_values(rows, fmt, rope)
        x = s["x"].double()
        if fmt == BF16:
            x = x.float().to(torch.bfloat16).double()
        else:
            b = x[:, :LATENT].reshape(-1, 32)
            unit = torch.ldexp(torch.ones_like(b[:, :1]), torch.frexp(b.abs().amax(1, keepdim=True))[1] - 3)  # a logarithm can fall below an exact power of two
            y = b / unit
            # the spacing of e2m1 at each magnitude: 1/2 below 2, 1 below 4, 2 above; round() takes ties to even
            step = torch.where(y.abs() < 2, 0.5, torch.where(y.abs() < 4, 1.0, 2.0))
            y = (torch.round(y / step) * step).clamp(-6, 6) * unit
            x = torch.cat([y.reshape(-1, LATENT), x[:, LATENT:].float().to(torch.bfloat16).double()], 1)
        if case["back"]:
            return x
        pool = s["pool"].view(torch.bfloat16).double().reshape(-1, LATENT + rope)
        pool[s["slots"]] = x
        return pool.reshape(s["pool"].shape[0], -1)
    if op == "attend":
        outs, lses = [], []
        rows = case["rows"]
        step = max(1, min(rows, (1 << 28) // (max(case["top"], 1 if case["mode"] == "top" else case["hi"]) * (LATENT + case["rope"]))))
        records, table = s["pool"].view(-1, _record(case["fmt"], case["rope"])), s["page_table"].long()
        for a in range(0, rows, step):
            n = s["row_len"][a:a + step].long()
            at = s["idx"][a:a + step].long() if s["idx"] is not None else torch.arange(int(n.max()), device=n.device).repeat(n.numel(), 1)
            dead = (at < 0) | (at >= n[:, None])
            at = at.masked_fill(dead, 0)
            own_pages = table[torch.zeros_like(n) if case["shared"] else torch.arange(a, a + n.numel(), device=n.device)]
            k = _exact_values(records[(torch.gather(own_pages, 1, at // PAGE) * PAGE + at % PAGE).reshape(-1)], case["fmt"], case["rope"]).reshape(*at.shape, -1)
            z = torch.einsum("bhd,bnd->bhn", s["q"][a:a + step].double(), k) * s["scale"]
            z = z.masked_fill(dead[:, None, :], -math.inf)
            lses.append(torch.logsumexp(z, 2))
            outs.append(torch.einsum("bhn,bnd->bhd", torch.softmax(z, 2), k[..., :LATENT]))
        return {"out": torch.cat(outs), "lse": torch.cat(lses)}
    outs, lses = [], []
    qs, ks = s["q_start"].tolist(), s["kv_start"].tolist()
    for r in range(case["requests"]):
        q, kn, v = s["q"][qs[r]:qs[r + 1]].double(), s["k_nope"][ks[r]:ks[r + 1]].double(), s["v"][ks[r]:ks[r + 1]].double()
        kr = s["k_rope"][ks[r]:ks[r + 1]].double()
        lq, lk = q.shape[0], kn.shape[0]
        hidden = torch.ones(lq, lk, dtype=torch.bool, device=q.device).triu(lk - lq + 1)
        z = torch.einsum("ihd,jhd->hij", q[..., :NOPE], kn) + torch.einsum("ihd,jd->hij", q[..., NOPE:], kr)
        z = (z * s["scale"]).masked_fill(hidden, -math.inf)
        lses.append(torch.logsumexp(z, 2).t())
        outs.append(torch.einsum("hij,jhd->ihd", torch.softmax(z, 2), v))
    return {"out": torch.cat(outs), "lse": torch.cat(lses)}
