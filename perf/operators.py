"""Cases for timing and checking the paged latent-cache operators and prefill attention.

Five operators, as a serving loop uses them:

  plan     block tables and slot maps for the tokens of a step, from request lengths (s4r_page_plan)
  write    latent rows into the pages of a cache, in bf16 or in 4 bits with group scales (s4r_latent_write)
  attend   attention of every head over one shared latent vector a token, absorbed form, from pages (s4r_latent_attend)
  project  per-head products between head space and latent space: absorbing queries, expanding keys, values and
           outputs (s4r_latent_project)
  prefill  causal attention over expanded keys and values of ragged prompts (s4r_prefill_attend)

`run` computes each in plain torch operations in 32 bits, or (own = True) through the library.
"""
import math

import torch

own = False

GROUP = 16           # values that share a scale in the 4-bit format
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one decode step of a busy server: 256 requests, a token each, some of them opening a page
        dict(name="plan_decode_256", op="plan", batch=256, page=64, low=1, high=8000, new_low=1, new_high=1, spare=500),
        # a step that admits prompts: ragged new tokens, small pages, a pool too small for the last requests
        dict(name="plan_admit_1001", op="plan", batch=1001, page=16, low=0, high=4100, new_low=0, new_high=1200, spare=-700),
        # the decode step's rows of a middle-sized batch
        dict(name="write_bf16_64", op="write", cache="bf16", n=64, width=576, page=64, rows=65536),
        # a prompt of 32K tokens into 4-bit pages
        dict(name="write_fp4_32k", op="write", cache="fp4", n=32765, width=576, page=64, rows=65536),
        # one request, 8K of context, 16 heads (a slice of the heads): latency counts
        dict(name="attend_bf16_1x8k_h16", op="attend", cache="bf16", batch=1, queries=1, heads=16, rank=512, rope=64,
             page=64, low=8191, high=8191),
        # an ordinary ragged decode batch
        dict(name="attend_bf16_32x8k_h64", op="attend", cache="bf16", batch=32, queries=1, heads=64, rank=512, rope=64,
             page=64, low=500, high=16000),
        # two tokens a request (a draft checked), all 128 heads, a long batch
        dict(name="attend_bf16_8x32k_h128_q2", op="attend", cache="bf16", batch=8, queries=2, heads=128, rank=512, rope=64,
             page=128, low=20001, high=44000),
        # the cache in 4 bits: a few requests up to 128K long, small pages, a number of heads that fills no tile
        dict(name="attend_fp4_5x128k_h20", op="attend", cache="fp4", batch=5, queries=1, heads=20, rank=512, rope=64,
             page=16, low=7, high=131068),
        # absorbing the queries of a decode step
        dict(name="project_absorb_64", op="project", to_latent=True, n=64, heads=128, dim=128, rank=512, shared=False),
        # expanding the keys of a prompt from its latents
        dict(name="project_expand_8k", op="project", to_latent=False, n=8190, heads=32, dim=128, rank=512, shared=True),
        # a prompt of 8K with the shared rotary part, and grouped heads with ragged lengths and a cached prefix
        dict(name="prefill_8k_h16", op="prefill", batch=1, hq=16, hkv=16, dim=128, rope=64, vdim=128, low=8192, high=8192,
             prefix=0),
        dict(name="prefill_ragged_gqa", op="prefill", batch=6, hq=32, hkv=8, dim=128, rope=0, vdim=128, low=33, high=2900,
             prefix=517),
    ]


def _logu(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["plan", "write", "attend", "attend", "attend", "project", "prefill", "prefill"])
    while True:
        if op == "plan":
            decode = rng.random() < 0.5
            c = dict(op=op, batch=_logu(rng, 1, 2000), page=rng.choice([16, 32, 64, 128]), low=rng.choice([0, 1, 17]),
                     high=_logu(rng, 20, 9000), new_low=1 if decode else 0, new_high=1 if decode else _logu(rng, 2, 4000),
                     spare=rng.choice([1000, 100, 0, -20]) + rng.randrange(20))
            total = c["batch"] * (c["new_low"] + c["new_high"]) / 2
            if total <= 600600 and c["batch"] * (c["high"] + c["new_high"]) / c["page"] <= 2 ** 20:
                return c
        elif op == "write":
            return dict(op=op, cache=rng.choice(["bf16", "fp4"]), n=_logu(rng, 1, 32000), width=32 * rng.randrange(4, 19),
                        page=rng.choice([16, 32, 64, 128]), rows=1024 * rng.randrange(32, 65))
        elif op == "attend":
            high = _logu(rng, 2, 100000)
            c = dict(op=op, cache=rng.choice(["bf16", "fp4"]), batch=_logu(rng, 1, 100), queries=rng.choice([1, 1, 1, 2, 3, 4]),
                     heads=_logu(rng, 4, 128), rank=64 * rng.randrange(2, 9), rope=rng.choice([0, 32, 64]),
                     page=rng.choice([16, 32, 64, 128]), low=rng.choice([0, 1, high // 2, high]), high=high)
            tokens = c["batch"] * (c["low"] + high) / 2
            if tokens <= 250000 and tokens * c["queries"] * c["heads"] <= 60e6:
                return c
        elif op == "project":
            lat = rng.random() < 0.5
            c = dict(op=op, to_latent=lat, n=_logu(rng, 1, 8000), heads=_logu(rng, 1, 128), dim=rng.choice([32, 64, 96, 128]),
                     rank=64 * rng.randrange(2, 9), shared=not lat and rng.random() < 0.5)
            if c["n"] * c["heads"] <= 250000:
                return c
        else:
            hkv = rng.choice([1, 2, 4, 8])
            high = _logu(rng, 2, 6000)
            c = dict(op=op, batch=_logu(rng, 1, 12), hq=hkv * rng.choice([1, 2, 3, 4]), hkv=hkv, dim=rng.choice([64, 128]),
                     rope=rng.choice([0, 64]), vdim=rng.choice([64, 128]), low=rng.choice([1, high // 2, high]), high=high,
                     prefix=rng.choice([0, 0, _logu(rng, 1, 3000)]))
            if c["batch"] * c["hq"] * c["high"] * (c["high"] + c["prefix"]) <= 1.0e9:
                return c


def _spread(n, low, high, phase=0.5):
    """n whole numbers from low to high, spread evenly in no order (golden ratio), the same for every seed."""
    low = max(0, min(low, high))
    return [low + int((phase + i * 0.6180339887498949) % 1.0 * (high - low + 1)) for i in range(n)]


def _cdiv(a, b):
    return -(-a // b)


def _plan_lengths(c):
    old = _spread(c["batch"], c["low"], c["high"])
    new = _spread(c["batch"], c["new_low"], c["new_high"], 0.25)
    return old, new


def _row_bytes(c, width):
    return width * 2 if c["cache"] == "bf16" else width * 9 // 16


def work(case):
    c = case
    if c["op"] == "plan":
        old, new = _plan_lengths(c)
        pages = sum(_cdiv(a + b, c["page"]) - _cdiv(a, c["page"]) for a, b in zip(old, new))
        pages = min(pages, max(0, pages + c["spare"]))
        # lengths and counts in, lengths and offsets out; an id read and an entry written a page; slot, position, request a token
        return {"bytes": 16.0 * c["batch"] + 8.0 * pages + 16.0 * sum(new), "flops": 0.0}
    if c["op"] == "write":
        stored = 2 * c["width"] if c["cache"] == "fp4" else 0
        return {"bytes": float(c["n"]) * (2 * c["width"] + 8 + _row_bytes(c, c["width"]) + stored), "flops": 0.0}
    if c["op"] == "attend":
        lens = _spread(c["batch"], c["low"], c["high"])
        width, rows = c["rank"] + c["rope"], c["batch"] * c["queries"] * c["heads"]
        seen = sum(max(0, n - c["queries"] + 1 + t) for n in lens for t in range(c["queries"]))
        return {"bytes": float(sum(lens) * _row_bytes(c, width) + rows * 2 * (width + c["rank"]) + rows * 4),
                "flops": 2.0 * seen * c["heads"] * (width + c["rank"])}
    if c["op"] == "project":
        wide = c["heads"] * c["dim"]
        x = c["rank"] if c["shared"] else (wide if c["to_latent"] else c["heads"] * c["rank"])
        y = c["heads"] * c["rank"] if c["to_latent"] else wide
        return {"bytes": 2.0 * (c["n"] * (x + y) + wide * c["rank"]), "flops": 2.0 * c["n"] * wide * c["rank"]}
    lens = _spread(c["batch"], c["low"], c["high"])
    q, k = sum(lens), sum(n + c["prefix"] for n in lens)
    seen = sum(n * c["prefix"] + n * (n + 1) // 2 for n in lens)
    return {"bytes": 2.0 * (q * c["hq"] * (c["dim"] + c["rope"] + c["vdim"]) + k * (c["hkv"] * (c["dim"] + c["vdim"]) + c["rope"]))
            + 4.0 * q * c["hq"],
            "flops": 2.0 * seen * c["hq"] * (c["dim"] + c["rope"] + c["vdim"])}


# ------------------------------------------------------------------ inputs

def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _tables(g, counts, width):
    """Block tables [len(counts)][width] with counts[b] pages each, pages in random order, -1 behind them; and the page count."""
    total = sum(counts)
    order = torch.randperm(max(1, total), generator=g, device="cuda").to(torch.int32)
    n = _i32(counts)
    first = (torch.cumsum(n, 0) - n)[:, None]
    col = torch.arange(width, device="cuda", dtype=torch.int32)[None]
    at = (first + col).clamp(max=max(0, total - 1)).long()
    return torch.where(col < n[:, None], order[at], torch.full_like(col, -1)).contiguous(), max(1, total)


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    s = {"case": c, "kept": {}}
    if c["op"] == "plan":
        old, new = _plan_lengths(c)
        # other seeds: the same lengths in another order of the requests
        shift = int(torch.randint(0, 1 << 30, (1,), generator=g, device="cuda")) % c["batch"]
        old, new = old[shift:] + old[:shift], new[shift:] + new[:shift]
        page = c["page"]
        have = [_cdiv(a, page) for a in old]
        need = sum(_cdiv(a + b, page) for a, b in zip(old, new)) - sum(have)
        width = max(1, max(_cdiv(a + b, page) for a, b in zip(old, new)))
        free = max(0, need + c["spare"])
        total = sum(have) + free
        order = torch.randperm(max(1, total), generator=g, device="cuda").to(torch.int32)
        n = _i32(have)
        col = torch.arange(width, device="cuda", dtype=torch.int32)[None]
        at = ((torch.cumsum(n, 0) - n)[:, None] + col).clamp(max=max(0, total - 1)).long()
        s["table"] = torch.where(col < n[:, None], order[at], torch.full_like(col, -1)).contiguous()
        s["free_pages"] = torch.cat([order[sum(have):total], torch.zeros(8, dtype=torch.int32, device="cuda")])
        s["free_count"] = _i32([free])
        s["lengths"], s["new"] = _i32(old), _i32(new)
        tokens = sum(new)
        s["lengths_out"], s["free_out"] = torch.empty_like(s["lengths"]), torch.empty_like(s["free_count"])
        s["cu"] = torch.empty(c["batch"] + 1, dtype=torch.int32, device="cuda")
        s["slots"] = torch.empty(tokens + 5, dtype=torch.int64, device="cuda")
        s["positions"] = torch.empty(tokens + 5, dtype=torch.int32, device="cuda")
        s["requests"] = torch.empty(tokens + 5, dtype=torch.int32, device="cuda")
    elif c["op"] == "write":
        pages = c["rows"] // c["page"]
        s["latents"] = _randn(g, c["n"], c["width"]).to(torch.bfloat16)
        s["slots"] = torch.randperm(pages * c["page"], generator=g, device="cuda")[: c["n"]].contiguous()
        if c["n"] > 3:
            s["slots"][c["n"] // 2] = -1     # a padded token
        if c["cache"] == "bf16":
            s["cache"] = torch.zeros(pages, c["page"], c["width"], dtype=torch.bfloat16, device="cuda")
        else:
            s["cache"] = torch.zeros(pages, c["page"] * c["width"] * 9 // 16, dtype=torch.uint8, device="cuda")
            s["stored"] = torch.zeros(c["n"], c["width"], dtype=torch.bfloat16, device="cuda")
    elif c["op"] == "attend":
        width = c["rank"] + c["rope"]
        lens = _spread(c["batch"], c["low"], c["high"])
        cols = max(1, _cdiv(c["high"], c["page"]))
        s["table"], pages = _tables(g, [_cdiv(n, c["page"]) for n in lens], cols)
        s["lengths"] = _i32(lens)
        rows = _randn(g, pages * c["page"], width).to(torch.bfloat16)
        s["q"] = _randn(g, c["batch"], c["queries"], c["heads"], width).to(torch.bfloat16)
        s["scale"] = 1.5 / math.sqrt(width)
        if c["cache"] == "bf16":
            s["cache"] = rows.view(pages, c["page"], width)
        else:
            s["cache"] = torch.zeros(pages, c["page"] * width * 9 // 16, dtype=torch.uint8, device="cuda")
            _store_fp4(s["cache"], c["page"], width, rows, torch.arange(pages * c["page"], device="cuda"))
        s["out"] = torch.empty(c["batch"], c["queries"], c["heads"], c["rank"], dtype=torch.bfloat16, device="cuda")
        s["lse"] = torch.empty(c["batch"], c["queries"], c["heads"], dtype=torch.float32, device="cuda")
    elif c["op"] == "project":
        d_in, d_out = (c["dim"], c["rank"]) if c["to_latent"] else (c["rank"], c["dim"])
        shape = (c["n"], d_in) if c["shared"] else (c["n"], c["heads"], d_in)
        s["x"] = _randn(g, *shape).to(torch.bfloat16)
        s["basis"] = (_randn(g, c["heads"] * c["dim"], c["rank"]) / math.sqrt(d_in)).to(torch.bfloat16)
        s["out"] = torch.empty(c["n"], c["heads"], d_out, dtype=torch.bfloat16, device="cuda")
    else:
        lens = _spread(c["batch"], c["low"], c["high"])
        cq, ck = [0], [0]
        for n in lens:
            cq.append(cq[-1] + n)
            ck.append(ck[-1] + n + c["prefix"])
        s["cu_q"], s["cu_k"], s["max_q"], s["max_k"] = _i32(cq), _i32(ck), max(lens), max(lens) + c["prefix"]
        s["q"] = _randn(g, cq[-1], c["hq"], c["dim"] + c["rope"]).to(torch.bfloat16)
        s["k"] = _randn(g, ck[-1], c["hkv"], c["dim"]).to(torch.bfloat16)
        s["k_rope"] = _randn(g, ck[-1], c["rope"]).to(torch.bfloat16) if c["rope"] else None
        s["v"] = _randn(g, ck[-1], c["hkv"], c["vdim"]).to(torch.bfloat16)
        s["scale"] = 1.5 / math.sqrt(c["dim"] + c["rope"])
        s["out"] = torch.empty(cq[-1], c["hq"], c["vdim"], dtype=torch.bfloat16, device="cuda")
        s["lse"] = torch.empty(cq[-1], c["hq"], dtype=torch.float32, device="cuda")
    return s


# ------------------------------------------------------------------ plain forms

def _codes(t):
    """4-bit codes (sign, then 2 exponent bits and 1 mantissa bit) of values already divided by their scale; ties to even."""
    a = t.abs()
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75).to(torch.uint8) + (a > 1.25).to(torch.uint8) + (a >= 1.75).to(torch.uint8)
            + (a > 2.5).to(torch.uint8) + (a >= 3.5).to(torch.uint8) + (a > 5.0).to(torch.uint8))
    return code + 8 * torch.signbit(t).to(torch.uint8)


def _values(codes):
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=torch.float32, device=codes.device)
    return table[codes.long()]


def _quantise(rows):
    """Rows [n][width] as codes, e4m3 scales and the values they stand for."""
    n, width = rows.shape
    t = rows.to(torch.float32).view(n, width // GROUP, GROUP)
    six = torch.full((), 6.0, device=t.device)       # on the device: a quotient, not a product with 1 / 6
    scale = (t.abs().amax(2) / six).clamp(max=448.0).to(torch.float8_e4m3fn)
    s = scale.to(torch.float32)[..., None]
    code = torch.where(s > 0, _codes(t / torch.where(s > 0, s, torch.ones_like(s))), torch.zeros_like(t, dtype=torch.uint8))
    return code.view(n, width), scale.view(torch.uint8), (_values(code) * s).view(n, width)


def _store_fp4(cache, page, width, rows, slots):
    """Quantises rows into the pages of a 4-bit cache (a page: its rows' codes, two a byte, then its rows' scales)."""
    code, scale, values = _quantise(rows)
    packed = code[:, 0::2] | (code[:, 1::2] << 4)
    half, part = page * width // 2, width // GROUP
    at, row = slots // page, slots % page
    flat = cache.view(cache.shape[0], -1)
    flat[:, :half].view(cache.shape[0], page, width // 2)[at, row] = packed
    flat[:, half:].view(cache.shape[0], page, part)[at, row] = scale
    return values


def _load_fp4(cache, page, width):
    """All rows of a 4-bit cache [pages * page][width] as values."""
    pages, half = cache.shape[0], page * width // 2
    packed = cache[:, :half].reshape(pages * page, width // 2)
    scale = cache[:, half:].reshape(pages * page, width // GROUP).view(torch.float8_e4m3fn).to(torch.float32)
    code = torch.stack([packed & 15, packed >> 4], 2).view(pages * page, width // GROUP, GROUP)
    return (_values(code) * scale[..., None]).view(pages * page, width)


def _plain_plan(s):
    c = s["case"]
    page, batch = c["page"], c["batch"]
    old, new, table = s["lengths"].long(), s["new"].long(), s["table"]
    width = table.shape[1]
    fits = (old >= 0) & (new >= 0) & (old + new <= width * page)
    have = (old + page - 1) // page
    need = torch.where(fits, (old + new + page - 1) // page - have, 0)
    upto = torch.cumsum(need, 0)
    free = s["free_count"].long()[0]
    served = fits & ((need == 0) | (upto <= free))
    taken = (need * served).sum()
    col = torch.arange(width, device=old.device)[None]
    fresh = served[:, None] & (col >= have[:, None]) & (col < (have + need)[:, None])
    at = (free - 1 - ((upto - need)[:, None] + col - have[:, None])).clamp(0, s["free_pages"].numel() - 1)
    full = torch.where(fresh, s["free_pages"][at], table)
    count = new.clamp(min=0)
    ends = torch.cumsum(count, 0)
    cu = torch.cat([torch.zeros_like(ends[:1]), ends])
    t = torch.arange(s["slots"].numel(), device=old.device)
    live = t < ends[-1]
    req = torch.searchsorted(ends, t, right=True).clamp(max=batch - 1)
    pos = old[req] + t - cu[req]
    pid = full[req, (pos // page).clamp(0, width - 1)].long()
    ok = live & served[req]
    minus = torch.full_like(t, -1)
    return {"table": full, "lengths": torch.where(served, old + new, old).int(), "free": (free - taken).int().view(1),
            "cu": cu.int(), "slots": torch.where(ok, pid * page + pos % page, minus),
            "positions": torch.where(live, pos, minus).int(), "requests": torch.where(live, req, minus).int()}


def _plain_write(s):
    c = s["case"]
    rows = s["latents"]
    keep = s["slots"] >= 0
    if c["cache"] == "bf16":
        flat = s["cache"].view(-1, c["width"])
        # a padded token writes back what its stand-in row holds
        at = torch.where(keep, s["slots"], s["slots"].amax())
        flat[at] = torch.where(keep[:, None], rows, rows[s["slots"].argmax()][None])
        return {"cache": s["cache"]}
    at = torch.where(keep, s["slots"], s["slots"].amax())
    put = torch.where(keep[:, None], rows, rows[s["slots"].argmax()][None])
    _store_fp4(s["cache"], c["page"], c["width"], put, at)
    return {"cache": s["cache"], "stored": _quantise(rows)[2].to(torch.bfloat16)}


def _plain_attend(s):
    c = s["case"]
    width, page, rank = c["rank"] + c["rope"], c["page"], c["rank"]
    rows = s["cache"].view(-1, width) if c["cache"] == "bf16" else _load_fp4(s["cache"], page, width)
    table = s["table"].long()
    longest = table.shape[1] * page
    pos = torch.arange(longest, device=table.device)
    at = table.clamp(min=0)[:, pos // page] * page + pos % page
    kv = rows[at].to(torch.float32)                                          # [batch][longest][width]
    q = s["q"].to(torch.float32)
    sees = s["lengths"].long()[:, None] - c["queries"] + 1 + torch.arange(c["queries"], device=table.device)[None]
    mask = pos[None, None] < sees[..., None]                                 # [batch][queries][longest]
    logit = torch.einsum("bthd,bld->bthl", q, kv) * s["scale"]
    logit = logit.masked_fill(~mask[:, :, None], -math.inf)
    top = logit.amax(3, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = torch.exp(logit - top)
    total = p.sum(3, keepdim=True)
    out = torch.einsum("bthl,bld->bthd", p, kv[..., :rank]) / torch.where(total > 0, total, torch.ones_like(total))
    return {"out": out.to(torch.bfloat16), "lse": (top + torch.log(total))[..., 0]}


def _plain_project(s):
    c = s["case"]
    x = s["x"].to(torch.float32)
    basis = s["basis"].to(torch.float32).view(c["heads"], c["dim"], c["rank"])
    form = "nhd,hdr->nhr" if c["to_latent"] else ("nr,hdr->nhd" if c["shared"] else "nhr,hdr->nhd")
    return torch.einsum(form, x, basis).to(torch.bfloat16)


def _padded(rows, cu, longest):
    """Ragged rows [total][...] as [batch][longest][...] (rows behind a sequence's end repeat some row) and their validity."""
    n = (cu[1:] - cu[:-1]).long()
    col = torch.arange(longest, device=cu.device)[None]
    at = (cu[:-1].long()[:, None] + col).clamp(max=rows.shape[0] - 1)
    return rows[at], col < n[:, None], at


def _plain_prefill(s):
    c = s["case"]
    group = c["hq"] // c["hkv"]
    q, q_ok, q_at = _padded(s["q"].to(torch.float32), s["cu_q"], s["max_q"])
    k, k_ok, _ = _padded(s["k"].to(torch.float32), s["cu_k"], s["max_k"])
    v = _padded(s["v"].to(torch.float32), s["cu_k"], s["max_k"])[0]
    b, mq = q.shape[:2]
    q = q.view(b, mq, c["hkv"], group, -1)
    logit = torch.einsum("bqgjd,bkgd->bgjqk", q[..., : c["dim"]], k)
    if c["rope"]:
        r = _padded(s["k_rope"].to(torch.float32), s["cu_k"], s["max_k"])[0]
        logit += torch.einsum("bqgjd,bkd->bgjqk", q[..., c["dim"]:], r)
    nq, nk = (s["cu_q"][1:] - s["cu_q"][:-1]), (s["cu_k"][1:] - s["cu_k"][:-1])
    last = (nk - nq)[:, None] + torch.arange(mq, device=q.device)[None]
    mask = k_ok[:, None] & (torch.arange(s["max_k"], device=q.device)[None, None] <= last[..., None])
    logit = logit.mul_(s["scale"]).masked_fill_(~mask[:, None, None], -math.inf)
    top = logit.amax(4, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = torch.exp(logit.sub_(top))
    total = p.sum(4, keepdim=True)
    o = torch.einsum("bgjqk,bkgd->bqgjd", p, v)
    o = o / torch.where(total > 0, total, torch.ones_like(total))[..., 0].permute(0, 3, 1, 2)[..., None]
    lse = (top + torch.log(total))[..., 0].permute(0, 3, 1, 2).reshape(b, mq, c["hq"])
    out = torch.empty_like(s["out"])
    flat = torch.empty_like(s["lse"])
    out[q_at[q_ok]] = o.reshape(b, mq, c["hq"], c["vdim"])[q_ok].to(torch.bfloat16)
    flat[q_at[q_ok]] = lse[q_ok]
    return {"out": out, "lse": flat}


def run(state):
    op = state["case"]["op"]
    if own:
        return _OWN[op](state)
    return {"plan": _plain_plan, "write": _plain_write, "attend": _plain_attend, "project": _plain_project,
            "prefill": _plain_prefill}[op](state)


# ------------------------------------------------------------------ the library's calls

def _own_plan(s):
    import rank_decode_attention_b200 as s4r
    s4r.s4r_page_plan(lengths=s["lengths"], new_tokens=s["new"], block_table=s["table"], free_pages=s["free_pages"],
                      free_count=s["free_count"], lengths_out=s["lengths_out"], free_count_out=s["free_out"],
                      cu_tokens=s["cu"], slots=s["slots"], positions=s["positions"], requests=s["requests"],
                      page_size=s["case"]["page"])
    return {"table": s["table"], "lengths": s["lengths_out"], "free": s["free_out"], "cu": s["cu"], "slots": s["slots"],
            "positions": s["positions"], "requests": s["requests"]}


def _own_write(s):
    import rank_decode_attention_b200 as s4r
    stored = s.get("stored")
    s4r.s4r_latent_write(latents=s["latents"], slots=s["slots"], cache=s["cache"], page_size=s["case"]["page"], stored=stored)
    return {"cache": s["cache"]} if stored is None else {"cache": s["cache"], "stored": stored}


def _own_attend(s):
    import rank_decode_attention_b200 as s4r
    kept = s["kept"]
    if "workspace" not in kept:     # a serving loop keeps its workspace
        a = s4r.latent_attend_args(q=s["q"], cache=s["cache"], block_table=s["table"], lengths=s["lengths"], out=s["out"],
                                   lse=s["lse"], page_size=s["case"]["page"], scale=s["scale"])
        kept["workspace"] = torch.empty(s4r.s4r_latent_attend_workspace_bytes(a), dtype=torch.uint8, device="cuda")
        s4r.s4r_workspace_init(kept["workspace"])
    s4r.s4r_latent_attend(s4r.latent_attend_args(
        q=s["q"], cache=s["cache"], block_table=s["table"], lengths=s["lengths"], out=s["out"], lse=s["lse"],
        page_size=s["case"]["page"], scale=s["scale"], workspace=kept["workspace"]))
    return {"out": s["out"], "lse": s["lse"]}


def _own_project(s):
    import rank_decode_attention_b200 as s4r
    s4r.s4r_latent_project(s["x"], s["basis"], s["out"], to_latent=s["case"]["to_latent"])
    return s["out"]


def _own_prefill(s):
    import rank_decode_attention_b200 as s4r
    s4r.s4r_prefill_attend(s4r.prefill_attend_args(
        q=s["q"], k=s["k"], v=s["v"], k_rope=s["k_rope"], cu_q=s["cu_q"], cu_k=s["cu_k"], max_q=s["max_q"], scale=s["scale"],
        out=s["out"], lse=s["lse"]))
    return {"out": s["out"], "lse": s["lse"]}


_OWN = {"plan": _own_plan, "write": _own_write, "attend": _own_attend, "project": _own_project, "prefill": _own_prefill}


# ------------------------------------------------------------------ exact values

def exact(case, seed):
    """The computed outputs from their definitions in 64 bits; None for whole numbers and copies."""
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "plan":
        return None
    if c["op"] == "write":
        if c["cache"] == "bf16":
            return None
        # nearest representable value to each x / scale on the signed grid; ties to the even code
        x = s["latents"].double().view(c["n"], -1, GROUP)
        scale = (x.abs().amax(2) / 6).float().clamp(max=448.0).to(torch.float8_e4m3fn).double()[..., None]
        grid = torch.tensor(E2M1, dtype=torch.float64, device=x.device)
        dist = (x.abs() / scale)[..., None] - grid
        even = torch.arange(8, device=x.device) % 2
        near = (dist.abs() * 2 ** 30).round() * 2 + even
        return {"cache": None, "stored": (grid[near.argmin(-1)] * torch.where(x < 0, -1.0, 1.0) * scale).view(c["n"], c["width"])}
    if c["op"] == "attend":
        width = c["rank"] + c["rope"]
        lens = s["lengths"].tolist()
        out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
        lse = torch.full(s["lse"].shape, -math.inf, dtype=torch.float64, device="cuda")
        for b, n in enumerate(lens):
            pages = s["table"][b, : _cdiv(n, c["page"])].long()
            if not n:
                continue
            if c["cache"] == "bf16":
                kv = s["cache"][pages].reshape(-1, width)[:n].double()
            else:
                raw = s["cache"][pages]
                half = c["page"] * width // 2
                nib = raw[:, :half].reshape(-1, width // 2).long()
                mag = torch.tensor(E2M1, dtype=torch.float64, device="cuda")
                lo, hi = nib % 16, nib // 16
                both = torch.stack([lo, hi], -1).view(-1, width)
                val = mag[both % 8] * (1 - 2 * (both // 8)).double()
                sc = raw[:, half:].reshape(-1, width // GROUP).view(torch.float8_e4m3fn).double()
                kv = (val * sc.repeat_interleave(GROUP, 1))[:n]
            for t in range(c["queries"]):
                m = n - c["queries"] + 1 + t
                if m <= 0:
                    continue
                z = s["q"][b, t].double() @ kv[:m].T * s["scale"]
                lse[b, t] = torch.logsumexp(z, 1)
                out[b, t] = torch.exp(z - lse[b, t][:, None]) @ kv[:m, : c["rank"]]
        return {"out": out, "lse": lse}
    if c["op"] == "project":
        basis = s["basis"].double().view(c["heads"], c["dim"], c["rank"])
        out = torch.empty(s["out"].shape, dtype=torch.float64, device="cuda")
        for h in range(c["heads"]):
            x = (s["x"] if c["shared"] else s["x"][:, h]).double()
            out[:, h] = x @ (basis[h] if c["to_latent"] else basis[h].T)
        return out
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["lse"].shape, -math.inf, dtype=torch.float64, device="cuda")
    cq, ck = s["cu_q"].tolist(), s["cu_k"].tolist()
    group = c["hq"] // c["hkv"]
    for b in range(c["batch"]):
        nq, nk = cq[b + 1] - cq[b], ck[b + 1] - ck[b]
        if not nq or not nk:
            continue
        late = torch.arange(nk, device="cuda")[None] > torch.arange(nq, device="cuda")[:, None] + nk - nq
        for h in range(c["hq"]):
            q = s["q"][cq[b]:cq[b + 1], h].double()
            k = s["k"][ck[b]:ck[b + 1], h // group].double()
            if c["rope"]:
                k = torch.cat([k, s["k_rope"][ck[b]:ck[b + 1]].double()], 1)
            z = (q @ k.T * s["scale"]).masked_fill_(late, -math.inf)
            lse[cq[b]:cq[b + 1], h] = torch.logsumexp(z, 1)
            out[cq[b]:cq[b + 1], h] = torch.exp(z - torch.logsumexp(z, 1)[:, None]) @ s["v"][ck[b]:ck[b + 1], h // group].double()
    return {"out": out, "lse": lse}
