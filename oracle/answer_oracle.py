"""Oracle of the calls between a denoising step's logits and the next step:
sampling, unmasking, and the runs of sequences that share pages. numpy,
float64, row by row; shares no code with the library.
"""
import math

import numpy as np


def sample_row(x, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """(token, log-probability) of one row of logits x (any float type)."""
    x = np.array(x, dtype=np.float64)
    x[np.isnan(x)] = -np.inf
    m = x.max()
    if m == -np.inf:
        return -1, -np.inf
    if m == np.inf:
        x = np.where(x == np.inf, 0.0, -np.inf)
        m = 0.0
    whole = math.log(np.exp(x - m).sum())  # above m, which may be so large that it would swallow it
    if not temperature >= 2.0 ** -20:
        got = int(np.flatnonzero(x == m)[0])
        return got, -whole
    t = min(float(temperature), 2.0 ** 40)
    ranked = sorted(range(x.size), key=lambda i: (-x[i], i)) if x.size < 64 else np.argsort(-x, kind="stable")
    ranked = np.asarray(ranked)
    if 0 < top_k < x.size:
        ranked = ranked[:int(top_k)]
    with np.errstate(over="ignore"):
        gap = (x[ranked] - m) / t
    w = np.exp(gap)
    if top_p < 1:
        before = np.concatenate([[0.0], np.cumsum(w)[:-1]])
        keep = before < max(float(top_p), 0.0) * w.sum()
        keep[0] = True
        ranked, w, gap = ranked[keep], w[keep], gap[keep]
    if min_p > 0:
        keep = gap >= math.log(min(float(min_p), 1.0))
        ranked, w = ranked[keep], w[keep]
    # weights are multiples of 2^-44: only where u is 1 does it show that the smallest ones are nothing
    ranked, w = ranked[w >= 2.0 ** -45], w[w >= 2.0 ** -45]
    order = np.argsort(ranked)
    ranked, sums = ranked[order], np.cumsum(w[order])
    hit = np.flatnonzero(sums > min(max(float(u), 0.0), 1.0) * sums[-1])
    got = int(ranked[hit[0]]) if hit.size else int(ranked[-1])
    return got, float(x[got] - m - whole)


def unmask(tokens, sampled, logprob, cu_rows, mask_id, n_min, threshold):
    """(tokens, left); n_min and threshold one per sequence. Rows behind the last offset stay. A drawn mask is no token."""
    out, left = np.array(tokens), []
    for s in range(len(cu_rows) - 1):
        rows = [i for i in range(cu_rows[s], cu_rows[s + 1]) if tokens[i] == mask_id]
        can = [i for i in rows if sampled[i] >= 0 and sampled[i] != mask_id]
        rank = sorted(can, key=lambda i: (math.isnan(logprob[i]), -logprob[i] if not math.isnan(logprob[i]) else 0.0, i))
        keep = {i for i in can if logprob[i] >= threshold[s]}
        if len(keep) < n_min[s]:
            keep = set(rank[:max(0, n_min[s])])
        for i in keep:
            out[i] = sampled[i]
        left.append(len(rows) - len(keep))
    return out, np.array(left)


def alike(table, lens, rows, page, pos=None):
    """(numbers of the sequences with rows, pages that each and the next begin with alike below the rows of both)."""
    busy = [s for s in range(len(rows)) if rows[s]]
    full = [max(0, min(lens[s], lens[s] - rows[s] if pos is None else pos[s])) // page for s in range(len(rows))]
    c = []
    for a, b in zip(busy, busy[1:]):
        n = 0
        while n < min(full[a], full[b]) and table[a][n] == table[b][n]:
            n += 1
        c.append(n)
    return busy, c


def runs(busy, c, n, page, longest=256):
    """int [3, n]: the cut that saves most, as bdlm_cache_prefixes writes it."""
    m = len(busy)
    best, came = [0] * (m + 1), [0] * (m + 1)
    for j in range(1, m + 1):
        low, top = None, None
        for i in range(j - 1, max(0, j - longest) - 1, -1):
            if i < j - 1:
                low = c[i] if low is None else min(low, c[i])
            got = best[i] + (j - 1 - i) * (low or 0)
            if top is None or got > top:  # of equal ones the shortest run stays
                top, came[j] = got, i
        best[j] = top
    plan = np.array([[s for s in range(n)], [s + 1 for s in range(n)], [0] * n])
    j = m
    while j > 0:
        i = came[j]
        shared = min(c[i:j - 1]) if j - i > 1 else 0
        if shared:
            plan[:, busy[i]:busy[j - 1] + 1] = np.array([[busy[i]], [busy[j - 1] + 1], [shared * page]])
        j = i
    return plan


def saved(plan, rows, page):
    """What a plan saves, in pages."""
    total = 0
    for s in range(len(rows)):
        if plan[0][s] == s and plan[2][s]:
            total += (sum(1 for i in range(s, plan[1][s]) if rows[i]) - 1) * (int(plan[2][s]) // page)
    return total
