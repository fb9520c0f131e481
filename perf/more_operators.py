"""Cases of the operators between a denoising step's last layer and the next step: what is timed, and their plain forms.

Several candidates answer the same prompt block by block. Their sequences share the prompt's pages of the 8-bit cache
(bdlm_cache_fork), attention reads what they share once for all of them, the step's logits become tokens, and the rows
that the model is surest of are kept.

  prefixes  which neighbouring sequences read which pages together (bdlm_cache_prefixes)
  attn      attention of new rows over the cache, a run's shared pages read once (bdlm_cache_attn_shared_fwd)
  sample    a token and its log-probability for each row of logits, from given random numbers (bdlm_sample)
  unmask    the rows of every block that keep their tokens in this step (bdlm_unmask)
"""
import math
import random

import torch

own = False

E4M3_MAX = 448.0
LONGEST_RUN = 256  # sequences
GREEDY_BELOW = 2.0 ** -20  # temperatures


# ----------------------------------------------------------------- the cases
def listed():
    return [
        # the smallest call: one token each for four candidates of a short prompt, a small model's heads
        {"name": "attn_token_4x1000", "op": "attn", "prompts": 1, "kids_lo": 4, "kids_hi": 4, "prefix_lo": 1000, "prefix_hi": 1000, "tail_lo": 1,
         "tail_hi": 40, "rows_lo": 1, "rows_hi": 1, "heads": 16, "kv_heads": 4, "d": 64, "page": 16, "block": 1, "spread": 1},
        # one token each for 64 candidates of one long prompt
        {"name": "attn_token_64x32k", "op": "attn", "prompts": 1, "kids_lo": 64, "kids_hi": 64, "prefix_lo": 32768, "prefix_hi": 32768, "tail_lo": 1,
         "tail_hi": 1024, "rows_lo": 1, "rows_hi": 1, "heads": 32, "kv_heads": 8, "d": 128, "page": 64, "block": 1, "spread": 2},
        # ragged: eleven prompts of one to nine candidates, odd row counts, three query heads per kv head, small pages
        {"name": "attn_ragged_11x9", "op": "attn", "prompts": 11, "kids_lo": 1, "kids_hi": 9, "prefix_lo": 5, "prefix_hi": 9001, "tail_lo": 1,
         "tail_hi": 701, "rows_lo": 0, "rows_hi": 23, "heads": 12, "kv_heads": 4, "d": 64, "page": 16, "block": 16, "spread": 3},
        # one denoising step: eight candidates each of eight prompts, blocks of 32 rows
        {"name": "attn_block32_8x8", "op": "attn", "prompts": 8, "kids_lo": 8, "kids_hi": 8, "prefix_lo": 4096, "prefix_hi": 32768, "tail_lo": 32,
         "tail_hi": 512, "rows_lo": 32, "rows_hi": 32, "heads": 32, "kv_heads": 8, "d": 128, "page": 128, "block": 32, "spread": 4},
        # 64 streams under one system prompt, four candidates of each document
        {"name": "prefixes_64", "op": "prefixes", "prompts": 16, "kids_lo": 4, "kids_hi": 4, "system": 2048, "prefix_lo": 1024, "prefix_hi": 16384,
         "tail_lo": 32, "tail_hi": 512, "rows_lo": 32, "rows_hi": 32, "page": 64, "block": 32, "spread": 5},
        # many streams, small pages, runs of all lengths, some streams idle
        {"name": "prefixes_600", "op": "prefixes", "prompts": 120, "kids_lo": 1, "kids_hi": 9, "system": 333, "prefix_lo": 1, "prefix_hi": 30912,
         "tail_lo": 1, "tail_hi": 2048, "rows_lo": 0, "rows_hi": 8, "page": 16, "block": 8, "spread": 6},
        # the smallest sampling: one token of one stream, everything on
        {"name": "sample_1x32001", "op": "sample", "rows": 1, "vocab": 32001, "dtype": "float32", "pad": 0, "temperature": 0.8, "top_k": 40,
         "top_p": 0.95, "min_p": 0.02, "head": 13.0, "masked": 0.0, "idle": 0.0, "spread": 7},
        # a denoising step of 16 streams, 32 rows each, of which every fourth has its token already
        {"name": "sample_16x32", "op": "sample", "rows": 512, "vocab": 131072, "dtype": "bfloat16", "pad": 0, "temperature": 1.0, "top_k": 0,
         "top_p": 0.95, "min_p": 0.0, "head": 13.0, "masked": 0.0, "idle": 0.25, "spread": 8},
        # plain sampling without filters from flat logits, an odd vocabulary whose rows are not aligned, a third of it masked
        {"name": "sample_flat_96", "op": "sample", "rows": 96, "vocab": 65537, "dtype": "float16", "pad": 2, "temperature": 1.25, "top_k": 0,
         "top_p": 1.0, "min_p": 0.0, "head": 0.0, "masked": 0.3, "idle": 0.0, "spread": 9},
        # requests of every kind in one batch: greedy, temperatures, top-k, top-p and min-p by row
        {"name": "sample_mixed_1024", "op": "sample", "rows": 1024, "vocab": 131072, "dtype": "bfloat16", "pad": 0, "temperature": -1.0, "top_k": -1,
         "top_p": -1.0, "min_p": -1.0, "head": 11.0, "masked": 0.0, "idle": 0.0, "spread": 10},
        # the rows of 16 blocks that keep their tokens
        {"name": "unmask_16x32", "op": "unmask", "seqs": 16, "rows_lo": 32, "rows_hi": 32, "masked": 0.75, "n_min": 4, "threshold": -0.1, "spread": 11},
        # many ragged blocks, a number and a threshold for each
        {"name": "unmask_700", "op": "unmask", "seqs": 700, "rows_lo": 0, "rows_hi": 1024, "masked": 0.5, "n_min": -1, "threshold": -1.0, "spread": 12},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "sample", "sample", "sample", "prefixes", "unmask"])
    c = {"op": op, "spread": rng.randrange(1 << 30)}
    if op == "sample":
        c["vocab"] = _log(rng, 1, 200000)
        c["rows"] = _log(rng, 1, max(1, min(1024, (1 << 26) // c["vocab"])))
        c["dtype"] = rng.choice(["bfloat16", "bfloat16", "float16", "float32"])
        c["pad"] = rng.choice([0, 0, 1, 7, 8])
        c["temperature"] = rng.choice([0.0, 1.0, -1.0, round(rng.uniform(0.2, 2.0), 3)])
        c["top_k"] = rng.choice([0, -1, 1, _log(rng, 1, c["vocab"]), _log(rng, 1, 200)])
        c["top_p"] = rng.choice([1.0, -1.0, 0.9, round(rng.uniform(0.01, 0.999), 4)])
        c["min_p"] = rng.choice([0.0, 0.0, -1.0, 0.05, round(rng.uniform(0.0001, 0.5), 5)])
        c["head"] = rng.choice([0.0, 8.0, 13.0, rng.uniform(2.0, 18.0)])
        c["masked"] = rng.choice([0.0, 0.0, 0.3, 0.999])
        c["idle"] = rng.choice([0.0, 0.0, 0.5])
        return c
    if op == "unmask":
        c["seqs"] = _log(rng, 1, 700)
        c["rows_hi"] = _log(rng, 1, 1024)
        c["rows_lo"] = rng.randint(0, c["rows_hi"])
        c["masked"] = rng.choice([1.0, 0.5, rng.random()])
        c["n_min"] = rng.choice([-1, 0, 1, rng.randint(1, 100)])
        c["threshold"] = rng.choice([-1.0, -0.01, -0.7, round(rng.uniform(-5.0, 0.0), 3)])
        return c
    c["page"] = rng.choice([16, 32, 64, 128])
    c["prompts"] = _log(rng, 1, 12 if op == "attn" else 120)
    c["kids_hi"] = _log(rng, 1, 64 // c["prompts"] + 1 if op == "attn" else 9)
    if op == "prefixes":
        c["prompts"], c["kids_hi"] = c["prompts"] + 2, c["kids_hi"] + 2
    c["kids_lo"] = rng.randint(1, c["kids_hi"])
    c["block"] = rng.choice([1, 4, 16, 32, rng.randint(2, 50)])
    c["rows_hi"] = rng.choice([1, min(32, c["block"]), rng.randint(1, 32)])
    c["rows_lo"] = rng.choice([c["rows_hi"], rng.randint(0, c["rows_hi"])])
    c["prefix_hi"] = _log(rng, 1, 32768 if c["prompts"] < 4 else 8192)
    c["prefix_lo"] = rng.randint(1, c["prefix_hi"])
    c["tail_hi"] = max(c["rows_hi"], _log(rng, 1, 1000))
    c["tail_lo"] = rng.randint(1, c["tail_hi"])
    if op == "prefixes":
        c["prefix_hi"] += 20 * c["page"]
        c["system"] = rng.choice([0, _log(rng, 1, 4000)])
        return c
    c["kv_heads"] = rng.choice([1, 2, 3, 4, 8])
    c["heads"] = c["kv_heads"] * rng.choice([1, 2, 3, 4, 5, 7, 8])
    c["d"] = rng.choice([64, 128])
    return c


def _pages(n, page):
    return -(-n // page)


def _streams(case):
    """The sequences of a case, from it alone: (prompt, pages shared with the prompt's others, length, new rows) of each."""
    rng, p, got = random.Random(case["spread"]), case["page"], []
    for i in range(case["prompts"]):
        n = case.get("system", 0) + min(case["prefix_hi"], max(case["prefix_lo"], _log(rng, case["prefix_lo"], case["prefix_hi"])))
        for _ in range(rng.randint(case["kids_lo"], case["kids_hi"])):
            r = rng.randint(case["rows_lo"], case["rows_hi"])
            tail = max(r, rng.randint(case["tail_lo"], case["tail_hi"]))
            if case["rows_lo"] == case["rows_hi"] == case["block"]:
                tail += -(n + tail) % case["block"]  # a denoising step: exactly the rows of one block
            got.append((i, n // p, n + tail, r))
    if not any(r for _, _, _, r in got):
        i, shared, n, _ = got[0]
        got[0] = i, shared, n + 1, 1
    return got


def _runs_of(case):
    """(first sequence, behind the last, shared positions) of every sequence, for the attention: the candidates of a prompt."""
    streams, p, runs = _streams(case), case["page"], []
    for i in range(case["prompts"]):
        mine = [s for s, x in enumerate(streams) if x[0] == i]
        busy = [s for s in mine if streams[s][3]]
        for s in mine:
            if len(busy) > 1 and streams[s][1] and busy[0] <= s <= busy[-1]:
                runs.append((busy[0], busy[-1] + 1, streams[s][1] * p))
            else:
                runs.append((s, s + 1, 0))
    return runs


def _blocks(case):
    """Rows, least number and threshold of every sequence of an unmask case."""
    rng, got = random.Random(case["spread"]), []
    for _ in range(case["seqs"]):
        r = rng.randint(case["rows_lo"], case["rows_hi"])
        got.append((r, rng.randint(0, max(1, r // 4)) if case["n_min"] < 0 else case["n_min"],
                    -10.0 * rng.random() ** 3 if case["threshold"] == -1.0 else case["threshold"]))
    if not any(r for r, _, _ in got):
        got[0] = (1,) + got[0][1:]
    return got


def _busy(case):
    """Which rows of a sampling case still lack their token."""
    rng = random.Random(case["spread"])
    return [not (rng.random() < case["idle"]) or i == 0 for i in range(case["rows"])]


def _visible(case, n, r):
    """Sum over the last r of n rows of the keys that each sees."""
    b, at, total = case["block"], n - r, 0
    while at < n:
        end = min(n, (at // b + 1) * b)
        total += (end - at) * end
        at = end
    return total


def work(case):
    if case["op"] == "sample":
        n, size = sum(_busy(case)), 4 if case["dtype"] == "float32" else 2
        return {"bytes": n * (case["vocab"] * size + 12) + 4 * case["rows"] * (case["idle"] > 0), "flops": 2 * n * case["vocab"]}
    if case["op"] == "unmask":
        blocks = _blocks(case)
        return {"bytes": 16 * sum(r for r, _, _ in blocks) + 16 * len(blocks), "flops": 0}
    streams, p = _streams(case), case["page"]
    if case["op"] == "prefixes":
        entries, busy = 0, [x for x in streams if x[3]]
        for i, x in enumerate(busy):  # a table row is read up to where it leaves its neighbours
            near = [y for y in busy[max(0, i - 1):i + 2] if y is not x]
            entries += max([(x[1] if x[0] == y[0] else case["system"] // p) + 1 for y in near] or [0])
        return {"bytes": 4 * (entries + 5 * len(streams)), "flops": 0}
    hk, h, d, keys, scales, flops, rows, seen = case["kv_heads"], case["heads"], case["d"], 0, 0, 0, 0, set()
    for (_, _, n, r), (first, _, shared) in zip(streams, _runs_of(case)):
        if r:
            own_keys = n - (shared if first in seen else 0)
            seen.add(first)
            keys += own_keys
            scales += _pages(own_keys, p)
            rows += r
            flops += _visible(case, n, r)
    return {"bytes": keys * hk * 2 * d + scales * (8 * hk + 4) + rows * h * (4 * d + 4), "flops": 4 * d * h * flops}


# ---------------------------------------------------------------- the inputs
def _scale_of(amax):
    """The smallest power of two s with amax / s <= 448 (1 where amax is 0)."""
    m, e = torch.frexp(amax)
    e = torch.where(m <= 0.875, e - 9, e - 8).clamp(min=-126)
    return torch.where(amax > 0, torch.ldexp(torch.ones_like(amax), e), torch.ones_like(amax))


def _pool(case, total, gen):
    """One layer's `total` pages: e4m3 keys and values [1, pages, Hk, page, d] and their scales."""
    hk, p, d, got = case["kv_heads"], case["page"], case["d"], []
    for gain in (2.0, 0.5):
        codes = torch.empty((total, hk, p, d), dtype=torch.float8_e4m3fn, device="cuda")
        scales = torch.empty((total, hk), dtype=torch.float32, device="cuda")
        step = max(1, (1 << 27) // (hk * p * d))
        for at in range(0, total, step):
            n = min(step, total - at)
            x = torch.randn((n, hk, p, d), generator=gen, device="cuda")
            x *= gain * torch.exp2(torch.randn((n, hk, 1, 1), generator=gen, device="cuda"))  # pages of unlike magnitude
            f = _scale_of(x.abs().amax((2, 3)))
            codes[at:at + n] = (x / f[:, :, None, None]).to(torch.float8_e4m3fn)
            scales[at:at + n] = f
        got += [codes[None], scales[None]]
    return got


def _int(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _float(v):
    return torch.tensor(v, dtype=torch.float32, device="cuda")


def _offsets(rows):
    at = [0]
    for r in rows:
        at.append(at[-1] + r)
    return at


def _prepare_cache(case, seed, gen):
    streams, p, rng = _streams(case), case["page"], random.Random(seed)
    n, system = len(streams), case.get("system", 0) // case["page"]
    if case["op"] == "prefixes":  # some branched off early
        streams = [x if rng.random() < 0.75 else (x[0], rng.randint(system, x[1]), x[2], x[3]) for x in streams]
    common, total, at_prompt, at_own = system, system, {}, []
    for i in range(case["prompts"]):
        at_prompt[i] = total
        total += max(x[1] for x in streams if x[0] == i) - common
    for _, shared, length, _ in streams:
        at_own.append(total)
        total += _pages(length, p) - shared
    ids = list(range(total + total // 8 + 3))
    rng.shuffle(ids)
    table = torch.full((n, max(_pages(x[2], p) for x in streams)), -1, dtype=torch.int32)
    for s, (i, shared, length, _) in enumerate(streams):
        row = ids[:common] + ids[at_prompt[i]:at_prompt[i] + shared - common] + ids[at_own[s]:at_own[s] + _pages(length, p) - shared]
        table[s, :len(row)] = torch.tensor(row, dtype=torch.int32)
    rows = [x[3] for x in streams]
    s = {"case": case, "table": table.cuda(), "lens": _int([x[2] for x in streams]), "lens_host": [x[2] for x in streams],
         "rows_host": rows, "cu_host": _offsets(rows), "cu": _int(_offsets(rows)), "busy": _int([i for i, r in enumerate(rows) if r])}
    if case["op"] == "prefixes":  # one layer's pages of one head stand for the pool: only their numbers matter
        s["pool"] = {"kv_heads": 1, "d": 64, "page": p}
        s["k"], s["ks"], s["v"], s["vs"] = _pool(s["pool"], len(ids), gen)
        return s
    s["k"], s["ks"], s["v"], s["vs"] = _pool(case, len(ids), gen)
    s["runs_host"] = _runs_of(case)
    s["runs"] = _int(s["runs_host"]).t().contiguous()
    s["q"] = (1.5 * torch.randn((s["cu_host"][-1], case["heads"], case["d"]), generator=gen, device="cuda")).bfloat16()
    return s


def _logits(case, gen):
    """A background of all tokens, a few that stand out by about `head`, and where it is asked for masked ones. Rows differ
    in how sharp they are."""
    dtype, v = getattr(torch, case["dtype"]), case["vocab"]
    x = torch.empty((case["rows"], v + case["pad"]), dtype=dtype, device="cuda")[:, :v]
    step = max(1, (1 << 26) // v)
    for at in range(0, case["rows"], step):
        n = min(step, case["rows"] - at)
        y = torch.randn((n, v), generator=gen, device="cuda")
        y *= 1.2 * torch.exp2(torch.rand((n, 1), generator=gen, device="cuda"))
        if case["head"] > 0:
            some = torch.randint(v, (n, 64), generator=gen, device="cuda")
            much = case["head"] + 3.0 * torch.randn((n, 64), generator=gen, device="cuda")
            few = torch.exp2(6.0 * torch.rand((n, 1), generator=gen, device="cuda"))
            y.scatter_add_(1, some, torch.where(torch.arange(64, device="cuda") < few, much, 0.0))
        if case["masked"] > 0:
            gone = torch.rand((n, v), generator=gen, device="cuda") < case["masked"]
            y.masked_fill_(gone, -math.inf)
        x[at:at + n] = y.to(dtype)
    return x


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    if case["op"] in ("attn", "prefixes"):
        return _prepare_cache(case, seed, gen)
    rng = random.Random(seed)
    if case["op"] == "unmask":
        blocks = _blocks(case)
        at = _offsets([r for r, _, _ in blocks])
        masked = torch.rand(at[-1], generator=gen, device="cuda") < case["masked"]
        s = {"case": case, "cu_host": at, "cu": _int(at), "mask_id": 31999,
             "tokens": torch.where(masked, 31999, torch.randint(31999, (at[-1],), generator=gen, device="cuda")).to(torch.int32),
             "sampled": torch.randint(31999, (at[-1],), generator=gen, device="cuda", dtype=torch.int32),
             # log-probabilities as bf16 logits give them: many near 0, some equal
             "logprob": -(4.0 * torch.rand(at[-1], generator=gen, device="cuda") ** 4).bfloat16().float(),
             "n_min": _int([k for _, k, _ in blocks]) if case["n_min"] < 0 else case["n_min"],
             "threshold": _float([x for _, _, x in blocks]) if case["threshold"] == -1.0 else case["threshold"]}
        s["longest"] = max(r for r, _, _ in blocks)
        return s
    n = case["rows"]
    s = {"case": case, "logits": _logits(case, gen), "u": torch.rand(n, generator=gen, device="cuda"), "mask_id": 7,
         "token": torch.zeros(n, dtype=torch.int32, device="cuda"), "logprob": torch.zeros(n, device="cuda")}
    s["temperature"] = _float([rng.choice([0.0, 1.0, rng.uniform(0.3, 1.5)]) for _ in range(n)]) if case["temperature"] < 0 else case["temperature"]
    s["top_k"] = _int([rng.choice([0, 0, _log(rng, 1, 200)]) for _ in range(n)]) if case["top_k"] < 0 else case["top_k"]
    s["top_p"] = _float([rng.choice([1.0, rng.uniform(0.5, 0.99)]) for _ in range(n)]) if case["top_p"] < 0 else case["top_p"]
    s["min_p"] = _float([rng.choice([0.0, 0.0, rng.uniform(0.01, 0.2)]) for _ in range(n)]) if case["min_p"] < 0 else case["min_p"]
    s["busy"] = _busy(case)
    s["tokens"] = _int([7 if b else 8 for b in s["busy"]]) if case["idle"] > 0 else None
    return s


# ------------------------------------------------------------ the plain forms
def _lcp(s, a, b, most):
    """Pages that the sequences a[i], b[i] begin with alike, at most `most`."""
    same = (s["table"][a] == s["table"][b]) & (torch.arange(s["table"].shape[1], device="cuda") < most[:, None])
    return same.long().cumprod(1).sum(1)


def _plain_prefixes(s):
    """The best cut of the sequences that have rows into runs, by what it saves: for each run (sequences - 1) * shared pages."""
    n, busy, p = len(s["rows_host"]), s["busy"].long(), s["case"]["page"]
    m = busy.numel()
    full = ((s["lens"] - (s["cu"][1:] - s["cu"][:-1])) // p).long()
    c = torch.cat([_lcp(s, busy[:-1], busy[1:], torch.minimum(full[busy[:-1]], full[busy[1:]])), torch.zeros(1, dtype=torch.long, device="cuda")])
    best = torch.zeros(m + 1, dtype=torch.long, device="cuda")
    came, got = torch.zeros_like(best), torch.zeros_like(best)  # where the last run of the best cut of the first j begins; what it shares
    low = torch.full((m,), 1 << 40, dtype=torch.long, device="cuda")
    ids = torch.arange(m, device="cuda")
    for j in range(1, m + 1):
        lo = max(0, j - LONGEST_RUN)
        low[j - 1] = 0
        if j >= 2:
            low[j - 2] = 1 << 40
            torch.minimum(low[lo:j - 1], c[j - 2], out=low[lo:j - 1])
        key = ((best[lo:j] + (j - 1 - ids[lo:j]) * low[lo:j]) * (m + 1) + ids[lo:j]).max()  # of cuts as good, the shortest last run
        best[j], came[j] = key // (m + 1), key % (m + 1)
        got[j:j + 1] = low.gather(0, came[j:j + 1])
    mark = torch.zeros(m + 1, dtype=torch.bool, device="cuda")  # the ends of the best cut's runs
    mark[m] = True
    jump, hops = came.clone(), 1
    while hops <= m:
        mark |= torch.zeros_like(mark).index_put_((torch.where(mark, jump, m),), torch.ones((), dtype=torch.bool, device="cuda"))
        jump, hops = jump[jump], 2 * hops
    behind = torch.flip(torch.cummin(torch.flip(torch.where(mark[1:], ids + 1, m), (0,)), 0).values, (0,))  # of each: its run's end
    first, last, shared = busy[came[behind]], busy[behind - 1], got[behind] * p
    s_ids = torch.arange(n, device="cuda")
    at = torch.searchsorted(busy, s_ids, right=True) - 1  # the last sequence with rows up to this one
    inside = (at >= 0) & (s_ids <= last[at.clamp(min=0)]) & (shared[at.clamp(min=0)] > 0)
    at = at.clamp(min=0)
    return torch.stack([torch.where(inside, first[at], s_ids), torch.where(inside, last[at] + 1, s_ids + 1),
                        torch.where(inside, shared[at], 0)]).to(torch.int32)


def _plain_attn(s):
    """What a run shares is taken once for all its rows, what each sequence has of its own one after the other."""
    c, (t, h, d) = s["case"], s["q"].shape
    p, hk, b = c["page"], c["kv_heads"], c["block"]
    g = h // hk
    o = torch.zeros((t, h, d), dtype=torch.bfloat16, device="cuda")
    lse = torch.full((h, t), -math.inf, device="cuda")

    def keys(i, lo, n):
        ids = s["table"][i, lo // p:_pages(n, p)].long()
        return ((s[x][0][ids].float() * s[x + "s"][0][ids][:, :, None, None]).transpose(0, 1).reshape(hk, -1, d)[:, :n - lo] for x in "kv")

    def part(q, k, v, seen):
        r = q.shape[0]
        x = torch.matmul(q.float().transpose(0, 1).reshape(hk, g * r, d), k.transpose(1, 2)).mul_(1.0 / math.sqrt(d)).view(h, r, -1)
        if seen is not None:
            x.masked_fill_(torch.arange(x.shape[2], device="cuda") >= seen[:, None], -math.inf)
        m = x.amax(-1)
        x.sub_(m[..., None]).exp_()
        return m, x.sum(-1), torch.matmul(x.view(hk, g * r, -1), v).view(h, r, d)

    for i, (first, end, shared) in enumerate(s["runs_host"]):
        if i == first:
            lo, hi = s["cu_host"][i], s["cu_host"][end]
            head = part(s["q"][lo:hi], *keys(i, 0, shared), None) if shared else None
        n, r = s["lens_host"][i], s["rows_host"][i]
        if not r:
            continue
        a = s["cu_host"][i]
        at = torch.arange(n - r, n, device="cuda")
        m, z, y = part(s["q"][a:a + r], *keys(i, shared, n), ((at // b + 1) * b).clamp(max=n) - shared)
        if shared:
            m0, z0, y0 = (x[:, a - lo:a - lo + r] for x in head)
            top = torch.maximum(m, m0)
            w, w0 = (m - top).exp(), (m0 - top).exp()
            m, z, y = top, z * w + z0 * w0, y * w[..., None] + y0 * w0[..., None]
        o[a:a + r] = (y / z[..., None]).transpose(0, 1).bfloat16()
        lse[:, a:a + r] = m + z.log()
    return o, lse


def _by_row(x, lo, hi):
    return x[lo:hi, None] if isinstance(x, torch.Tensor) else x


def _plain_sample(s):
    """Weights in 64 bits: a token is where their sum passes a random number, and the sums are long."""
    c, x = s["case"], s["logits"]
    n, v = x.shape
    ids, step = torch.arange(v, device="cuda"), max(1, (1 << 25) // v)
    for lo in range(0, n, step):
        hi = min(n, lo + step)
        y = x[lo:hi].float()
        m = y.amax(1, keepdim=True)
        gap = y.double() - m.double()
        gap = torch.where(y == -math.inf, -math.inf, gap)
        t = s["temperature"]
        t = (t[lo:hi, None] if isinstance(t, torch.Tensor) else torch.full((hi - lo, 1), t, device="cuda")).double()
        greedy = t < GREEDY_BELOW
        scaled = gap / torch.where(greedy, 1.0, t)
        w = scaled.exp()
        order = torch.sort(y, dim=1, descending=True, stable=True).indices
        ws = w.gather(1, order)
        k, p, mp = (_by_row(s[name], lo, hi) for name in ("top_k", "top_p", "min_p"))
        k = torch.as_tensor(k, device="cuda")
        keep = (ids < torch.where((k > 0) & (k < v), k, v)).expand(hi - lo, v).clone()
        z = torch.where(keep, ws, 0.0).sum(1, keepdim=True)
        before = torch.nn.functional.pad(ws.cumsum(1)[:, :-1], (1, 0))
        p = torch.as_tensor(p, device="cuda", dtype=torch.float32).double()
        keep &= (before < p * z) | (p >= 1) | (ids == 0)
        mp = torch.as_tensor(mp, device="cuda", dtype=torch.float32).double()
        keep &= (scaled.gather(1, order) >= mp.clamp(max=1.0).log()) | (mp <= 0)
        keep &= ws > 0
        kept = torch.zeros_like(keep).scatter_(1, order, keep)
        sums = torch.where(kept, w, 0.0).cumsum(1)
        hit = kept & (sums > s["u"][lo:hi, None].double() * sums[:, -1:])
        got = torch.where(hit, ids, v).amin(1)
        got = torch.where(got == v, torch.where(kept, ids, -1).amax(1), got)
        got = torch.where(greedy[:, 0], torch.where((y == m) & (m > -math.inf), ids, v).amin(1), got)
        got = torch.where((m[:, 0] == -math.inf) | (got == v), -1, got)
        lp = gap.gather(1, got.clamp(min=0)[:, None])[:, 0] - gap.exp().sum(1).log()
        lp = torch.where(got < 0, -math.inf, lp).float()
        if s["tokens"] is None:
            s["token"][lo:hi], s["logprob"][lo:hi] = got.to(torch.int32), lp
        else:
            todo = s["tokens"][lo:hi] == s["mask_id"]
            s["token"][lo:hi] = torch.where(todo, got.to(torch.int32), s["token"][lo:hi])
            s["logprob"][lo:hi] = torch.where(todo, lp, s["logprob"][lo:hi])
    return s["token"], s["logprob"]


def _plain_unmask(s):
    n, total = len(s["cu_host"]) - 1, s["cu_host"][-1]
    rows = (s["cu"][1:] - s["cu"][:-1]).long()
    seq = torch.repeat_interleave(torch.arange(n, device="cuda"), rows, output_size=total)
    at = torch.arange(total, device="cuda") - s["cu"][:-1].long()[seq]
    masked = s["tokens"] == s["mask_id"]
    can = masked & (s["sampled"] >= 0)
    sure = torch.where(can, s["logprob"], -math.inf)
    grid = torch.full((n, s["longest"]), -math.inf, device="cuda")
    live = torch.zeros((n, s["longest"]), dtype=torch.bool, device="cuda")
    grid[seq, at], live[seq, at] = sure, can
    # by falling certainty, rows that cannot be kept last, ties by their order
    order = torch.sort(torch.where(live, grid.double(), -1e300), dim=1, descending=True, stable=True).indices
    place = torch.empty_like(order).scatter_(1, order, torch.arange(s["longest"], device="cuda").expand(n, -1))
    least, floor = s["n_min"], s["threshold"]
    least = least[:, None] if isinstance(least, torch.Tensor) else least
    floor = floor[:, None] if isinstance(floor, torch.Tensor) else floor
    keep = live & ((grid >= floor) | (place < least))
    kept = keep[seq, at]
    left = (torch.zeros(n, dtype=torch.long, device="cuda").index_add_(0, seq, (masked & ~kept).long()))
    return torch.where(kept, s["sampled"], s["tokens"]), left.to(torch.int32)


def run(state):
    s, op = state, state["case"]["op"]
    if own:
        return _run_own(s, op)
    return {"prefixes": _plain_prefixes, "attn": _plain_attn, "sample": _plain_sample, "unmask": _plain_unmask}[op](s)


def _run_own(s, op):
    import block_diffusion_lm_bdlm_gb300 as bd

    if op == "sample":
        return bd.bdlm_sample(s["logits"], s["u"], temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"], min_p=s["min_p"],
                              tokens=s["tokens"], mask_id=s["mask_id"], out=s["token"], logprob=s["logprob"])
    if op == "unmask":
        return bd.bdlm_unmask(s["tokens"], s["sampled"], s["logprob"], s["cu"], s["mask_id"], n_min=s["n_min"], threshold=s["threshold"])
    if "cache" not in s:  # the handle that a program keeps: names of the tensors above, nothing of their contents
        s["cache"] = bd.PageCache(s["k"], s["v"], s["ks"], s["vs"], s["table"], s["lens"])
    if op == "prefixes":
        return bd.bdlm_cache_prefixes(s["cache"], s["cu"])
    return bd.bdlm_cache_attn_shared_fwd(s["cache"], s["q"], s["cu"], s["case"]["block"], s["runs"])


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
    """Every sequence over all of its own table, as if nothing were shared."""
    lut, p, b, d, h, hk = _values(), case["page"], case["block"], case["d"], case["heads"], case["kv_heads"]
    t = s["q"].shape[0]
    o = torch.zeros((t, h, d), dtype=torch.float64, device="cuda")
    lse = torch.full((h, t), -math.inf, dtype=torch.float64, device="cuda")
    step = max(1, 4096 // p)
    for i, (n, r) in enumerate(zip(s["lens_host"], s["rows_host"])):
        if r == 0:
            continue
        a = s["cu_host"][i]
        q = s["q"][a:a + r].double().reshape(r, hk, h // hk, d).permute(1, 2, 0, 3)
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


def _exact_sample(case, s):
    """Row by row on sorted lists of the tokens that each filter leaves."""
    n = case["rows"]
    token, logprob = torch.zeros(n, dtype=torch.int64, device="cuda"), torch.zeros(n, dtype=torch.float64, device="cuda")
    at = lambda x, i: float(x[i]) if isinstance(x, torch.Tensor) else float(torch.tensor(x, dtype=torch.float32))
    how = {k: (s[k].cpu() if isinstance(s[k], torch.Tensor) else s[k]) for k in ("temperature", "top_k", "top_p", "min_p")}
    u = s["u"].double().cpu()
    for i in range(n):
        if not s["busy"][i]:
            continue
        x = s["logits"][i].double()
        ids = (x > -math.inf).nonzero()[:, 0]
        if ids.numel() == 0:
            token[i], logprob[i] = -1, -math.inf
            continue
        t, k, p, mp = (at(how[name], i) for name in ("temperature", "top_k", "top_p", "min_p"))
        whole = torch.logsumexp(x, 0)
        if t < GREEDY_BELOW:
            t, k = 1.0, 1
        ranked = ids[torch.argsort(-x[ids], stable=True)]
        if 0 < k < ranked.numel():
            ranked = ranked[:int(k)]
        w = torch.exp((x[ranked] - x[ranked[0]]) / t)
        if p < 1:
            sums = torch.cumsum(w, 0)
            count = 1 + int((sums[:-1] < p * sums[-1]).sum())
            ranked, w = ranked[:count], w[:count]
        if mp > 0:
            fine = (x[ranked] - x[ranked[0]]) / t >= math.log(min(mp, 1.0))
            ranked, w = ranked[fine], w[fine]
        ranked, w = ranked[w > 0], w[w > 0]
        by_id = torch.argsort(ranked)
        ranked, sums = ranked[by_id], torch.cumsum(w[by_id], 0)
        j = min(int((sums <= u[i].to(sums.device) * sums[-1]).sum()), ranked.numel() - 1)
        token[i], logprob[i] = ranked[j], x[ranked[j]] - whole
    return token.to(torch.int32), logprob


def exact(case, seed):
    if case["op"] in ("prefixes", "unmask"):
        return None  # these choose and count
    w = work(case)
    if case["op"] == "attn" and (w["flops"] > 3e12 or w["bytes"] > 4e9):
        return None
    return {"attn": _exact_attn, "sample": _exact_sample}[case["op"]](case, prepare(case, seed))
