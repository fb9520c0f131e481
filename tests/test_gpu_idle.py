"""Runs with sequences that have no rows: they save no reads, so whether a run is read together goes by the others.
(test_gpu_shared holds the bounds' reasons.)"""
import numpy as np
import pytest
import torch

from oracle import cache_oracle as co

import cache_util as cu
from test_gpu_shared import bd, dev, plan_of  # noqa: F401  (bd is a fixture)

pytestmark = pytest.mark.gpu


def attend(bd, c, rows, plan, block, G, seed=0, **kw):
    off = cu.offsets(rows)
    Hk, d = c["k"].shape[2], c["k"].shape[4]
    q = torch.from_numpy(np.random.default_rng(seed).standard_normal((int(off[-1]), Hk * G, d))).bfloat16().cuda()
    got = bd.bdlm_cache_attn_shared_fwd(cu.to_device(bd, c), q, dev(off), block, plan, check=True, **kw)
    return q, off, got


def forest(seed, prefix_pages, tails, own, *, page, Hk, d):
    """A cache of sequences with a prefix and a tail each (None: nothing, and no page that is ever read); the prefixes are one and
    the same, or each one's own. The table with one prefix for all comes as well."""
    heads = [s for s, t in enumerate(tails) if t is not None] if own else [0]
    c = cu.make(seed, lens=[prefix_pages * page] * len(heads) + [t or 0 for t in tails], page=page, Hk=Hk, d=d)
    from_, n = c["table"], len(tails)
    table = np.zeros((n, prefix_pages + max(co.pages_of(t or 0, page) for t in tails)), dtype=from_.dtype)
    for s, t in enumerate(tails):
        if t is not None:
            m = co.pages_of(t, page)
            table[s, :prefix_pages] = from_[heads.index(s) if own else 0, :prefix_pages]
            table[s, prefix_pages:prefix_pages + m] = from_[len(heads) + s, :m]
    c["table"], c["lens"] = table, np.array([prefix_pages * page + (t or 0) for t in tails])
    alike = table.copy()
    alike[:, :prefix_pages] = table[next(s for s, t in enumerate(tails) if t is not None), :prefix_pages]
    return c, alike


@pytest.mark.parametrize("idle", [0, 1, 6, 29, 100])
@pytest.mark.parametrize("busy,rows,G,together", [(2, 32, 4, False), (2, 64, 2, False), (3, 43, 3, False), (16, 1, 4, True), (16, 4, 4, True)])
def test_idle_sequences_do_not_make_a_run_gain(bd, idle, busy, rows, G, together):
    """The members' tables are unlike here, which the call does not look at: a run that is read together goes by the first one's
    table, one that is read alone by each one's own. Blocks that fill an MMA tile each gain nothing by one reading, however many
    sequences without rows lie between them (flat rows >= 128 for each); few rows of many sequences over a long prefix do (5120 keys
    for 15 of 16, against 256 of each of 16 * 32 / 16 + 0.053 * 256 tiles at most)."""
    page, prefix, d = 128, 40, 64
    many = ([rows] + [0] * idle) * (busy - 1) + [rows]
    c, alike = forest(idle, prefix, [64 if r else None for r in many], True, page=page, Hk=1, d=d)
    n = len(many)
    q, off, got = attend(bd, c, many, dev(plan_of(n, [(0, n, prefix)], page)), rows, G)
    if together:
        c["table"] = alike
    ref = co.attention(c, 0, q.double().cpu().numpy(), off, rows, d ** -0.5)
    cu.check_attention(*got, ref, f"{idle} idle")


@pytest.mark.parametrize("n,every", [(40, 13), (300, 2), (700, 3), (700, 350)])
@pytest.mark.parametrize("rows,G", [(1, 4), (3, 3), (33, 2)])
def test_long_runs_with_idle_sequences(bd, n, every, rows, G):
    """More sequences than a CTA looks over at once, of which every so-manieth has rows; the whole as one run and as it is found."""
    page, prefix, d = 16, 60, 64
    many = [rows if s % every == every // 2 else 0 for s in range(n)]
    c, _ = forest(n, prefix, [r + s % 7 if r else None for s, r in enumerate(many)], False, page=page, Hk=2, d=d)
    c["table"][:, :prefix] = c["table"][many.index(rows), :prefix]
    ref = None
    for plan in (dev(plan_of(n, [(0, n, prefix)], page)), bd.bdlm_cache_prefixes(cu.to_device(bd, c), dev(cu.offsets(many)), check=True)):
        q, off, got = attend(bd, c, many, plan, rows, G)
        ref = ref or co.attention(c, 0, q.double().cpu().numpy(), off, rows, d ** -0.5)
        cu.check_attention(*got, ref, f"{n} {every}")
