"""Cases of the paged 8-bit cache operators: what is timed, and their plain forms.

The operators serve a block diffusion model: the committed (clean) blocks of
every sequence lie in a paged cache of e4m3 keys and values with one power-of-
two scale per page and kv head, the rows of the block being denoised (or one
token, or a prompt) are written behind them, and attention reads the pages.

  write    quantise new key and value rows into the pages (bdlm_cache_write)
  attn     attention of new rows over the cache, block-causal (bdlm_cache_attn_fwd)
  reserve  take free pages for growing sequences (bdlm_cache_reserve)
  fork     candidates that share a parent's full pages (bdlm_cache_fork)
  compact  move the live pages to the front of the pool (bdlm_cache_compact)
"""
import math
import random

import torch

own = False

E4M3_MAX = 448.0


# ----------------------------------------------------------------- the cases
def listed():
    return [
        # one denoising step of 16 streams: each stream's block of 32 rows is written behind a few thousand tokens
        {"name": "write_block_16x32", "op": "write", "seqs": 16, "len_lo": 512, "len_hi": 8192, "rows_lo": 32, "rows_hi": 32,
         "kv_heads": 8, "d": 128, "page": 64, "block": 32, "spread": 1},
        # eight whole prompts of ragged lengths enter an empty cache
        {"name": "write_prompts_8x8k", "op": "write", "seqs": 8, "len_lo": 4096, "len_hi": 12288, "rows_lo": 12288, "rows_hi": 12288,
         "kv_heads": 8, "d": 128, "page": 128, "block": 1, "spread": 2},
        # the smallest call: one token of one stream over a short cache, a small model's heads
        {"name": "attn_token_1x600", "op": "attn", "seqs": 1, "len_lo": 600, "len_hi": 600, "rows_lo": 1, "rows_hi": 1,
         "heads": 16, "kv_heads": 4, "d": 64, "page": 16, "block": 1, "spread": 3},
        # one token each for 64 streams whose lengths are spread like the packed training documents
        {"name": "attn_token_64_packed", "op": "attn", "seqs": 64, "len_lo": 512, "len_hi": 30912, "rows_lo": 1, "rows_hi": 1,
         "heads": 32, "kv_heads": 8, "d": 128, "page": 64, "block": 1, "spread": 4},
        # one denoising step of the same 64 streams, 32 rows each
        {"name": "attn_block32_64_packed", "op": "attn", "seqs": 64, "len_lo": 512, "len_hi": 30912, "rows_lo": 32, "rows_hi": 32,
         "heads": 32, "kv_heads": 8, "d": 128, "page": 64, "block": 32, "spread": 4},
        # one denoising step of one stream at the long context, 64 rows
        {"name": "attn_block64_1x128k", "op": "attn", "seqs": 1, "len_lo": 131072, "len_hi": 131072, "rows_lo": 64, "rows_hi": 64,
         "heads": 32, "kv_heads": 8, "d": 128, "page": 128, "block": 64, "spread": 5},
        # ragged verification and denoising rows: odd row counts, three query heads per kv head, pages that end inside a tile
        {"name": "attn_ragged_37", "op": "attn", "seqs": 37, "len_lo": 1, "len_hi": 9001, "rows_lo": 1, "rows_hi": 47,
         "heads": 12, "kv_heads": 4, "d": 64, "page": 16, "block": 16, "spread": 6},
        # prompts: three whole prompts, block-causal, read back from the cache that they were just written to
        {"name": "attn_prompts_3x8k", "op": "attn", "seqs": 3, "len_lo": 5000, "len_hi": 9000, "rows_lo": 9000, "rows_hi": 9000,
         "heads": 32, "kv_heads": 8, "d": 128, "page": 128, "block": 32, "spread": 7},
        # room for the next block of 256 streams
        {"name": "reserve_256", "op": "reserve", "seqs": 256, "len_lo": 128, "len_hi": 16384, "rows_lo": 32, "rows_hi": 32,
         "kv_heads": 1, "d": 64, "page": 64, "block": 32, "layers": 1, "spread": 8},
        # four candidates of one stream
        {"name": "fork_1x4", "op": "fork", "seqs": 1, "kids": 4, "len_lo": 1000, "len_hi": 1000, "rows_lo": 1, "rows_hi": 1,
         "kv_heads": 8, "d": 128, "page": 64, "block": 32, "layers": 8, "spread": 9},
        # four candidates each of 32 streams, all layers of a model
        {"name": "fork_32x4", "op": "fork", "seqs": 32, "kids": 4, "len_lo": 200, "len_hi": 1500, "rows_lo": 1, "rows_hi": 1,
         "kv_heads": 8, "d": 128, "page": 128, "block": 32, "layers": 32, "spread": 10},
        # the pool is drawn together after most streams have ended
        {"name": "compact_48", "op": "compact", "seqs": 48, "len_lo": 64, "len_hi": 4096, "rows_lo": 1, "rows_hi": 1,
         "kv_heads": 8, "d": 128, "page": 64, "block": 32, "layers": 8, "slack": 3, "spread": 11},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "write", "write", "reserve", "fork", "compact"])
    hk = rng.choice([1, 2, 3, 4, 8])
    c = {"op": op, "kv_heads": hk, "d": rng.choice([64, 128]), "page": rng.choice([16, 32, 64, 128]),
         "block": rng.choice([1, 4, 16, 32, 64, rng.randint(2, 100)]), "spread": rng.randrange(1 << 30)}
    if op == "write":
        c["seqs"] = _log(rng, 1, 96)
        c["rows_hi"] = _log(rng, 1, 4096 * 8 // max(8, c["seqs"]))
        c["rows_lo"] = rng.randint(1, c["rows_hi"])
        c["len_lo"], c["len_hi"] = c["rows_lo"], max(c["rows_hi"], _log(rng, 1, 16384))
        return c
    if op == "attn":
        c["heads"] = hk * rng.choice([1, 2, 3, 4, 5, 7, 8])
        kind = rng.choice(["token", "block", "rows", "prompt"])
        if kind == "prompt":
            c["seqs"], c["len_hi"] = rng.randint(1, 3), _log(rng, 33, 4000)
            c["len_lo"] = rng.randint(1, c["len_hi"])
            c["rows_lo"] = c["rows_hi"] = c["len_hi"]
            return c
        c["seqs"] = _log(rng, 1, 96)
        c["len_hi"] = _log(rng, 2, min(120000, 300000 // c["seqs"]))
        c["len_lo"] = rng.randint(1, c["len_hi"])
        c["rows_hi"] = {"token": 1, "block": min(c["block"], 64), "rows": rng.randint(1, 64)}[kind]
        c["rows_lo"] = 1 if kind == "rows" else c["rows_hi"]
        return c
    c["seqs"] = _log(rng, 1, 300 if op == "reserve" else 40)
    c["len_hi"] = _log(rng, 1, 16384 if op == "reserve" else 2048)
    c["len_lo"] = rng.randint(1, c["len_hi"])
    c["rows_lo"], c["rows_hi"] = 0, rng.randint(1, 200)
    c["layers"] = 1 if op == "reserve" else rng.randint(1, 12)
    if op == "fork":
        c["kids"] = rng.randint(1, 5)
    if op == "compact":
        c["slack"] = rng.randint(2, 4)
    return c


def _lengths(case):
    """(lengths with the new rows, new rows) of every sequence; from the case alone."""
    rng = random.Random(case["spread"])
    lens, rows = [], []
    for _ in range(case["seqs"]):
        n = min(case["len_hi"], max(case["len_lo"], _log(rng, case["len_lo"], case["len_hi"])))
        r = rng.randint(case["rows_lo"], case["rows_hi"])
        if case["rows_lo"] == case["rows_hi"] == case["block"] and n > r:
            n -= n % case["block"]  # a denoising step: exactly the rows of one block
        lens.append(n)
        rows.append(min(r, n))
    return lens, rows


def _pages(n, page):
    return -(-n // page)


def _visible(case, n, r):
    """Sum over the rows of the keys that each sees."""
    b, at, total = case["block"], n - r, 0
    while at < n:
        end = min(n, (at // b + 1) * b)
        total += (end - at) * end
        at = end
    return total


def _pool_pages(case):
    """(pages in the pool, pages of each sequence, pages that lie behind the first `live` ones)."""
    lens, rows = _lengths(case)
    if case["op"] in ("reserve", "fork"):
        lens = [n - r if case["op"] == "reserve" else n for n, r in zip(lens, rows)]
    need = [_pages(n, case["page"]) for n in lens]
    live = sum(need)
    total = live * case["slack"] + 1 if case["op"] == "compact" else live + _pages(live, 8) + 3
    total += sum(_pages(r, case["page"]) + 1 for r in rows) if case["op"] == "reserve" else 0
    total += case["seqs"] * case["kids"] if case["op"] == "fork" else 0
    return total, need, live * (total - live) // total


def _placed(case, seed):
    """Where every sequence's pages lie: (pages in the pool, page lists of the sequences)."""
    total, need, behind = _pool_pages(case)
    rng, live = random.Random(seed), sum(need)
    ids = rng.sample(range(live), live - behind) + rng.sample(range(live, total), behind)
    rng.shuffle(ids)
    lists, at = [], 0
    for k in need:
        lists.append(ids[at:at + k])
        at += k
    return total, lists


def work(case):
    lens, rows = _lengths(case)
    hk, d, p, layers = case["kv_heads"], case["d"], case["page"], case.get("layers", 1)
    if case["op"] == "attn":
        h = case["heads"]
        keys = sum(n for n, r in zip(lens, rows) if r)
        scales = sum(_pages(n, p) for n, r in zip(lens, rows) if r)
        t = sum(rows)
        return {"bytes": keys * hk * 2 * d + scales * (8 * hk + 4) + t * h * (4 * d + 4),
                "flops": 4 * d * h * sum(_visible(case, n, r) for n, r in zip(lens, rows))}
    if case["op"] == "write":
        old = sum((n - r) % p for n, r in zip(lens, rows) if r)
        touched = sum((n - 1) // p - (n - r) // p + 1 for n, r in zip(lens, rows) if r)
        # new rows read in 16 bits and written in 8, the rows before them in a page read (they are rewritten only
        # where the page's scale changes), scales written
        return {"bytes": hk * (2 * d * (3 * sum(rows) + old) + 8 * touched), "flops": 0}
    if case["op"] == "reserve":
        grown = sum(_pages(n, p) - _pages(n - r, p) for n, r in zip(lens, rows))
        return {"bytes": 4 * (sum(_pages(n - r, p) for n, r in zip(lens, rows)) + grown + 3 * case["seqs"]), "flops": 0}
    if case["op"] == "fork":
        tails = sum(n % p for n in lens) * case["kids"]
        tables = sum(_pages(n, p) for n in lens) * (1 + case["kids"])
        return {"bytes": layers * tails * hk * 4 * d + 4 * tables, "flops": 0}
    _, need, moved = _pool_pages(case)
    return {"bytes": moved * layers * hk * (4 * p * d + 16) + 8 * sum(need), "flops": 0}


# ---------------------------------------------------------------- the inputs
def _scale_of(amax):
    """The smallest power of two s with amax / s <= 448 (1 where amax is 0, never below 2^-126)."""
    m, e = torch.frexp(amax)
    e = torch.where(m <= 0.875, e - 9, e - 8).clamp(min=-126)
    return torch.where(amax > 0, torch.ldexp(torch.ones_like(amax), e), torch.ones_like(amax))


def _pool(case, total, gen):
    """A pool of `total` pages per layer: e4m3 keys, values [layers, pages, Hk, page, d] and their scales."""
    layers, hk, p, d = case.get("layers", 1), case["kv_heads"], case["page"], case["d"]
    got = []
    for gain in (2.0, 0.5):
        codes = torch.empty((layers, total, hk, p, d), dtype=torch.float8_e4m3fn, device="cuda")
        scales = torch.empty((layers, total, hk), dtype=torch.float32, device="cuda")
        flat = codes.view(layers * total, hk, p, d)
        flats = scales.view(layers * total, hk)
        step = max(1, (1 << 27) // (hk * p * d))
        for at in range(0, layers * total, step):
            n = min(step, layers * total - at)
            x = torch.randn((n, hk, p, d), generator=gen, device="cuda")
            x *= gain * torch.exp2(torch.randn((n, hk, 1, 1), generator=gen, device="cuda"))  # pages of unlike magnitude
            s = _scale_of(x.abs().amax((2, 3)))
            flat[at:at + n] = (x / s[:, :, None, None]).to(torch.float8_e4m3fn)
            flats[at:at + n] = s
        got += [codes, scales]
    return got


def _int(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    lens, rows = _lengths(case)
    total, lists = _placed(case, seed)
    kids = case.get("kids", 0) * case["seqs"]
    wide = max(_pages(n, case["page"]) for n in lens) + (2 if case["op"] == "reserve" else 0)
    k, ks, v, vs = _pool(case, total, gen)
    table = torch.full((case["seqs"] + kids, wide), -1, dtype=torch.int32)
    for i, pages in enumerate(lists):
        table[i, :len(pages)] = torch.tensor(pages, dtype=torch.int32)
    s = {"case": case, "k": k, "v": v, "ks": ks, "vs": vs, "table": table.cuda(), "lens_host": lens, "rows_host": rows,
         "lens": _int(lens + [0] * kids)}
    at = [0]
    for r in rows:
        at.append(at[-1] + r)
    s["cu_host"], s["cu"] = at, _int(at)
    if case["op"] == "attn":
        s["q"] = (1.5 * torch.randn((at[-1], case["heads"], case["d"]), generator=gen, device="cuda")).bfloat16()
    if case["op"] == "write":
        shape = (at[-1], case["kv_heads"], case["d"])
        s["k_new"] = (2.0 * torch.randn(shape, generator=gen, device="cuda")).bfloat16()
        s["v_new"] = torch.randn(shape, generator=gen, device="cuda").bfloat16()
        s["touched"] = sum((n - 1) // case["page"] - (n - r) // case["page"] + 1 for n, r in zip(lens, rows) if r)
    if case["op"] == "reserve":
        s["old"] = _int([n - r for n, r in zip(lens, rows)])
        s["new"] = _int(lens)
        s["lens"] = s["old"].clone()
    if case["op"] == "fork":
        s["parents"] = _int([i for i in range(case["seqs"]) for _ in range(case["kids"])])
        s["children"] = _int(list(range(case["seqs"], case["seqs"] + kids)))
    if case["op"] == "compact":
        s["table_was"] = s["table"].clone()
    return s


# ------------------------------------------------------------ the plain forms
def _plain_attn(s):
    """One sequence after the other: their lengths differ by up to 60 times, so a padded batch would be mostly padding."""
    c, (t, h, d) = s["case"], s["q"].shape
    p, hk, b = c["page"], c["kv_heads"], c["block"]
    g = h // hk
    o = torch.zeros((t, h, d), dtype=torch.bfloat16, device="cuda")
    lse = torch.full((h, t), -math.inf, device="cuda")
    for i, (n, r) in enumerate(zip(s["lens_host"], s["rows_host"])):
        if not r:
            continue
        pages = s["table"][i, :_pages(n, p)].long()
        k, v = ((s[x][0][pages].float() * s[x + "s"][0][pages][:, :, None, None]).transpose(0, 1).reshape(hk, -1, d)[:, :n] for x in "kv")
        q = s["q"][s["cu_host"][i]:s["cu_host"][i + 1]].float().transpose(0, 1).reshape(hk, g * r, d)
        x = torch.matmul(q, k.transpose(1, 2)).mul_(1.0 / math.sqrt(d)).view(hk, g, r, n)
        at = torch.arange(n - r, n, device="cuda")
        end = ((at // b + 1) * b)[:, None]
        x.masked_fill_(torch.arange(n, device="cuda") >= end, -math.inf)
        m = x.amax(-1, keepdim=True)
        x.sub_(m).exp_()
        z = x.sum(-1, keepdim=True)
        y = torch.matmul(x.view(hk, g * r, n), v).view(hk, g, r, d) / z
        o[s["cu_host"][i]:s["cu_host"][i + 1]] = y.view(h, r, d).transpose(0, 1).bfloat16()
        lse[:, s["cu_host"][i]:s["cu_host"][i + 1]] = (m + z.log()).view(h, r)
    return o, lse


def _touched(s):
    """The pages that new rows fall into: (sequence, page id, position of each of their rows)."""
    c = s["case"]
    p, n = c["page"], s["lens"].long()
    r = (s["cu"][1:] - s["cu"][:-1]).long()
    first = (n - r) // p
    count = torch.where(r > 0, (n - 1) // p - first + 1, 0)
    seq = torch.repeat_interleave(torch.arange(c["seqs"], device="cuda"), count, output_size=s["touched"])
    j = torch.arange(s["touched"], device="cuda") - (count.cumsum(0) - count)[seq] + first[seq]
    pos = j[:, None] * p + torch.arange(p, device="cuda")
    return seq, s["table"][seq, j].long(), pos, (n - r)[seq][:, None], n[seq][:, None]


def _plain_write(s):
    seq, page, pos, start, end = _touched(s)
    new, old = (pos >= start) & (pos < end), pos < start
    row = torch.where(new, s["cu"][:-1].long()[seq][:, None] + pos - start, 0)
    for x in "kv":
        codes, scales = s[x][0], s[x + "s"][0]
        was = codes[page]
        y = s[x + "_new"][row].float().transpose(1, 2)  # [pages, Hk, page, d]
        y = torch.where(new[:, None, :, None], y, torch.where(old[:, None, :, None], was.float() * scales[page][:, :, None, None], 0.0))
        f = _scale_of(y.abs().amax((2, 3)))
        y = (y / f[:, :, None, None]).to(torch.float8_e4m3fn)
        keep = (new | old)[:, None, :, None].expand_as(y)
        codes.view(torch.uint8)[page] = torch.where(keep, y.view(torch.uint8), was.view(torch.uint8))
        scales[page] = f
    return s["k"], s["v"], s["ks"], s["vs"]


def _live(s):
    """Whether each page is named by a sequence's first ceil(length / page) entries."""
    used = torch.arange(s["table"].shape[1], device="cuda") < ((s["lens"] + s["case"]["page"] - 1) // s["case"]["page"])[:, None]
    mark = torch.zeros(s["k"].shape[1] + 1, dtype=torch.bool, device="cuda")
    mark[torch.where(used, s["table"], s["k"].shape[1]).long()] = True
    return used, mark[:-1]


def _plain_reserve(s):
    p = s["case"]["page"]
    s["lens"].copy_(s["old"])  # the last step's rows are dropped
    used, live = _live(s)
    free = torch.argsort(live.to(torch.int8), stable=True).to(torch.int32)  # the free pages first, ascending
    more = (torch.arange(s["table"].shape[1], device="cuda") < ((s["new"] + p - 1) // p)[:, None]) & ~used
    nth = more.reshape(-1).cumsum(0).reshape(more.shape) - 1
    s["table"].copy_(torch.where(more, free[nth.clamp(min=0)], s["table"]))
    s["lens"].copy_(s["new"])
    return s["table"], s["lens"]


def _plain_fork(s):
    p, kids = s["case"]["page"], s["children"].long()
    s["lens"][kids] = 0  # the last round's candidates are dropped
    _, live = _live(s)
    free = torch.argsort(live.to(torch.int8), stable=True)
    n = s["lens"][s["parents"].long()]
    tail = (n % p).long()
    dst = free[((tail > 0).cumsum(0) - 1).clamp(min=0)]
    row = s["table"][s["parents"].long()]
    at = torch.arange(row.shape[1], device="cuda")
    src = row.gather(1, (n // p).long().clamp(max=row.shape[1] - 1)[:, None])[:, 0].long()
    row = torch.where(at == (n // p)[:, None], dst[:, None].to(torch.int32), row)
    s["table"][kids] = torch.where(at < ((n + p - 1) // p)[:, None], row, s["table"][kids])
    s["lens"][kids] = n
    some = tail > 0
    src, dst, keep = src[some], dst[some], (torch.arange(p, device="cuda") < tail[some][:, None])[:, None, :, None]
    for x in "kv":
        codes = s[x].view(torch.uint8)
        codes[:, dst], s[x + "s"][:, dst] = torch.where(keep, codes[:, src], codes[:, dst]), s[x + "s"][:, src]
    return s["table"], s["lens"], s["k"], s["v"], s["ks"], s["vs"]


def _plain_compact(s):
    s["table"].copy_(s["table_was"])
    used, live = _live(s)
    count = live.sum()
    ids = torch.arange(live.numel(), device="cuda")
    holes, movers = (~live & (ids < count)).nonzero()[:, 0], (live & (ids >= count)).nonzero()[:, 0]
    to = ids.clone()
    to[movers] = holes
    for x in "kv":
        codes = s[x].view(torch.uint8)
        codes[:, holes], s[x + "s"][:, holes] = codes[:, movers], s[x + "s"][:, movers]
    s["table"].copy_(torch.where(used, to[s["table"].clamp(min=0).long()].to(torch.int32), s["table"]))
    return s["table"], count.to(torch.int32).view(1), s["k"], s["v"], s["ks"], s["vs"]


def run(state):
    s, op = state, state["case"]["op"]
    if own:
        return _run_own(s, op)
    return {"attn": _plain_attn, "write": _plain_write, "reserve": _plain_reserve, "fork": _plain_fork, "compact": _plain_compact}[op](s)


def _run_own(s, op):
    import block_diffusion_lm_bdlm_gb300 as bd

    if "cache" not in s:  # the handle that a program keeps: names of the tensors above, nothing of their contents
        s["cache"] = bd.PageCache(s["k"], s["v"], s["ks"], s["vs"], s["table"], s["lens"])
    if op == "attn":
        return bd.bdlm_cache_attn_fwd(s["cache"], s["q"], s["cu"], s["case"]["block"])
    if op == "write":
        bd.bdlm_cache_write(s["cache"], s["k_new"], s["v_new"], s["cu"])
        return s["k"], s["v"], s["ks"], s["vs"]
    if op == "reserve":
        s["lens"].copy_(s["old"])
        bd.bdlm_cache_reserve(s["cache"], s["new"])
        return s["table"], s["lens"]
    if op == "fork":
        s["lens"][s["case"]["seqs"]:] = 0
        bd.bdlm_cache_fork(s["cache"], s["parents"], s["children"])
        return s["table"], s["lens"], s["k"], s["v"], s["ks"], s["vs"]
    s["table"].copy_(s["table_was"])
    count = bd.bdlm_cache_compact(s["cache"])
    return s["table"], count, s["k"], s["v"], s["ks"], s["vs"]


# ------------------------------------------------- the definition, in 64 bits
def _values():
    """The 256 values of e4m3: sign, four exponent bits with bias 7, three mantissa bits."""
    got = []
    for c in range(256):
        e, m = c >> 3 & 15, c & 7
        x = math.ldexp(m, -9) if e == 0 else math.ldexp(8 + m, e - 10)
        got.append(math.nan if c & 127 == 127 else -x if c & 128 else x)
    return torch.tensor(got, dtype=torch.float64, device="cuda")


def _exact_attn(case, s):
    lut, p, b, d = _values(), case["page"], case["block"], case["d"]
    h, hk = case["heads"], case["kv_heads"]
    t = s["q"].shape[0]
    o = torch.zeros((t, h, d), dtype=torch.float64, device="cuda")
    lse = torch.full((h, t), -math.inf, dtype=torch.float64, device="cuda")
    step = max(1, 2048 // p)
    for i, (n, r) in enumerate(zip(s["lens_host"], s["rows_host"])):
        if r == 0:
            continue
        a = s["cu_host"][i]
        q = s["q"][a:a + r].double().reshape(r, hk, h // hk, d).permute(1, 2, 0, 3)  # [Hk, G, r, d]
        seen = torch.tensor([min(n, (x // b + 1) * b) for x in range(n - r, n)], device="cuda")
        top = torch.full((hk, h // hk, r), -math.inf, dtype=torch.float64, device="cuda")
        z, y = torch.zeros_like(top), torch.zeros(q.shape, dtype=torch.float64, device="cuda")
        for j in range(0, _pages(n, p), step):
            ids = s["table"][i, j:min(j + step, _pages(n, p))].long()
            kk, vv = (lut[s[x][0][ids].view(torch.uint8).long()] * s[x + "s"][0][ids].double()[:, :, None, None] for x in "kv")
            kk, vv = (x.permute(1, 0, 2, 3).reshape(hk, 1, -1, d) for x in (kk, vv))
            key = torch.arange(j * p, j * p + kk.shape[2], device="cuda")
            x = (q / math.sqrt(d)) @ kk.transpose(2, 3)
            x = torch.where(key < seen[:, None], x, -math.inf)
            now = torch.maximum(top, x.amax(-1))
            safe = torch.where(torch.isinf(now), 0.0, now)
            w, fade = torch.exp(x - safe[..., None]), torch.exp(top - safe)
            z, y, top = z * fade + w.sum(-1), y * fade[..., None] + w @ vv, now
        o[a:a + r] = (y / z[..., None]).permute(2, 0, 1, 3).reshape(r, h, d)
        lse[:, a:a + r] = (top + torch.log(z)).reshape(h, r)
    return o, lse


def _nearest(x, lut):
    """The e4m3 value nearest to each x (|x| <= 448); of two as near, the one of even code."""
    up = lut[:127].contiguous()
    a = x.abs()
    hi = torch.searchsorted(up, a).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    dl, dh = a - up[lo], up[hi] - a
    return torch.copysign(up[torch.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)], x)


def _exact_write(case, s):
    lut, p = _values(), case["page"]
    out = []
    for x in "kv":
        codes = lut[s[x][0].view(torch.uint8).long()]
        scales = s[x + "s"][0].double().clone()
        for i, (n, r) in enumerate(zip(s["lens_host"], s["rows_host"])):
            for j in range((n - r) // p, _pages(n, p) if r else 0):
                page, a, e = int(s["table"][i, j]), max(0, n - r - j * p), min(p, n - j * p)
                at = s["cu_host"][i] + j * p + a - (n - r)
                new = s[x + "_new"][at:at + e - a].double().transpose(0, 1)
                y = torch.cat([codes[page, :, :a] * scales[page][:, None, None], new], 1)
                big = y.abs().amax((1, 2))
                f = torch.exp2(torch.ceil(torch.log2(big / E4M3_MAX)))
                f = torch.where(big / f > E4M3_MAX, 2 * f, torch.where(2 * big / f <= E4M3_MAX, f / 2, f))
                f = torch.where(big > 0, f.clamp(min=2.0 ** -126), 1.0)
                codes[page, :, :e] = _nearest(y / f[:, None, None], lut)
                scales[page] = f
        out.append((codes[None], scales[None]))
    return out[0][0], out[1][0], out[0][1], out[1][1]


def exact(case, seed):
    if case["op"] not in ("attn", "write"):
        return None  # these move and count: whole values and copies
    w = work(case)
    if w["flops"] > 6e12 or w["bytes"] > 4e9:
        return None
    return {"attn": _exact_attn, "write": _exact_write}[case["op"]](case, prepare(case, seed))
