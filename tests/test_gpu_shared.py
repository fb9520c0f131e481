"""Runs of sequences that share pages, and attention that reads what they share once, on the GPU against the float64
oracles (cache_util holds the attention's error bounds; joining the two parts adds three roundings in fp32, 2^-22 of A,
which the bounds' 2^-12 for exponentials and sums covers, and 2^-22 of 1 + |lse|, which their 2^-20 covers)."""
import numpy as np
import pytest
import torch

from oracle import answer_oracle as ao
from oracle import cache_oracle as co

import cache_util as cu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def bd():
    import block_diffusion_lm_bdlm_gb300 as m

    m.load_library()
    return m


def dev(x, dtype=torch.int32):
    return torch.as_tensor(np.asarray(x)).to("cuda", dtype)


def tree(seed, lens, shares, *, page, Hk, d, **kw):
    """A cache in which shares = [(first, end, pages)] sequences name the first one's leading pages."""
    c = cu.make(seed, lens=lens, page=page, Hk=Hk, d=d, **kw)
    for a, b, n in shares:
        for s in range(a + 1, b):
            c["table"][s, :n] = c["table"][a, :n]
    return c


def plan_of(n, shares, page):
    p = np.array([[s for s in range(n)], [s + 1 for s in range(n)], [0] * n])
    for a, b, k in shares:
        p[:, a:b] = [[a], [b], [k * page]]
    return p


# ---------------------------------------------------------------------- runs
@pytest.mark.parametrize("seed", range(24))
def test_runs(bd, seed):
    rng = np.random.default_rng(seed)
    page, n = int(rng.choice([16, 32, 64, 128])), int(rng.integers(1, 60))
    wide = int(rng.choice([3, 40, 700]))
    table = np.full((n, wide), -1)
    table[0] = rng.permutation(5 * wide)[:wide]
    for s in range(1, n):  # each branches off one before it, mostly the last
        p = s - 1 if rng.random() < 0.8 else int(rng.integers(0, s))
        k = int(rng.integers(0, wide + 1)) if rng.random() < 0.7 else wide
        table[s] = np.concatenate([table[p][:k], rng.integers(0, 5 * wide, wide - k)])
    rows = rng.integers(0, 4, n) * (rng.random(n) < 0.8)
    lens = np.minimum(rows + rng.integers(0, wide * page, n), wide * page)
    cache = bd.PageCache.empty(1, 4, page, 1, 64, n, wide)
    cache.table.copy_(dev(table))
    cache.lens.copy_(dev(lens))
    busy, c = ao.alike(table, lens, rows, page)
    runs = bd.bdlm_cache_prefixes(cache, dev(cu.offsets(rows)), check=True)
    assert np.array_equal(runs.cpu().numpy(), ao.runs(busy, c, n, page))
    pos = np.maximum(0, lens - rng.integers(0, 3 * page, n))
    busy, c = ao.alike(table, lens, rows, page, pos)
    out = torch.full((3, n), -3, dtype=torch.int32, device="cuda")
    assert bd.bdlm_cache_prefixes(cache, dev(cu.offsets(rows)), q_pos=dev(pos), out=out) is out
    assert np.array_equal(out.cpu().numpy(), ao.runs(busy, c, n, page))


@pytest.mark.parametrize("n,wide", [(256, 9), (257, 9), (600, 5), (4000, 3), (16384, 2)])
def test_long_runs(bd, n, wide):
    """More sequences than a run holds, all alike or alike in stretches."""
    rng = np.random.default_rng(n)
    for groups in (1, n // 300 + 2):
        of = np.sort(rng.integers(0, groups, n))
        table = np.repeat(np.arange(groups), np.bincount(of, minlength=groups))[:, None] * wide + np.arange(wide)
        table[:, 0] = 0
        lens = np.full(n, wide * 16)
        cache = bd.PageCache.empty(1, 4, 16, 1, 64, n, wide)
        cache.table.copy_(dev(table))
        cache.lens.copy_(dev(lens))
        rows = np.ones(n, dtype=int)
        rows[rng.random(n) < 0.02] = 0
        busy, c = ao.alike(table, lens, rows, 16)
        runs = bd.bdlm_cache_prefixes(cache, dev(cu.offsets(rows)), check=True)
        assert np.array_equal(runs.cpu().numpy(), ao.runs(busy, c, n, 16))


@pytest.mark.parametrize("off,lens,bad", [([1, 2, 3], [40, 40], 0), ([0, 2, 1], [40, 40], 1), ([0, 1, 2], [40, 1000], 1),
                                          ([0, 1, 42], [40, 40], 1), ([0, 1, 2], [-1, 40], 0)])
def test_runs_of_malformed_calls(bd, off, lens, bad):
    cache = bd.PageCache.empty(1, 4, 16, 1, 64, 2, 3)
    cache.lens.copy_(dev(lens))
    ws = torch.zeros(1024, dtype=torch.uint8, device="cuda")
    runs = bd.bdlm_cache_prefixes(cache, dev(off), workspace=ws)
    assert bd.bdlm_read_error(ws) == 6 and ws.view(torch.int32)[1].item() == bad
    assert runs.tolist() == [[0, 1], [1, 2], [0, 0]]
    with pytest.raises(bd.BDLMError):
        bd.bdlm_cache_prefixes(cache, dev([0, 1, 2]), total_rows=1, check=True)


# ----------------------------------------------------------------- attention
CASES = [
    # lens (with the new rows), rows, shares, page, Hk, G, d, block
    ([40, 41], [1, 1], [(0, 2, 2)], 16, 1, 1, 64, 1),
    ([40, 41, 50, 90], [1, 1, 1, 1], [(0, 4, 2)], 16, 2, 4, 128, 1),
    ([300, 310, 400, 290], [20, 3, 0, 7], [(0, 4, 4)], 64, 2, 3, 64, 8),
    ([130, 130, 77, 200, 260, 260], [2, 2, 5, 1, 4, 4], [(0, 2, 1), (3, 6, 1)], 128, 1, 8, 128, 4),
    ([3000, 3100, 3300], [32, 32, 32], [(0, 3, 23)], 128, 2, 4, 128, 32),       # cut prefix units
    ([1500] * 9, [33] * 9, [(0, 9, 60)], 16, 1, 2, 64, 11),                      # more than one unit of rows
    ([200] * 70, [1] * 70, [(0, 35, 3), (35, 70, 2)], 32, 1, 5, 64, 1),
    ([2100, 2100, 64, 64, 2049, 2300], [1, 1, 64, 1, 1, 200], [(0, 2, 32), (4, 6, 16)], 64, 4, 1, 128, 64),
    ([48, 48], [16, 16], [(0, 2, 2)], 16, 2, 2, 64, 16),                         # nothing but the new rows behind the prefix
    ([500, 20, 33], [1, 1, 1], [], 16, 2, 2, 64, 1),                             # no run at all
    ([800] * 40 + [30], [1, 0, 2] * 13 + [1, 3], [(0, 40, 40)], 16, 3, 7, 128, 2),
]


@pytest.mark.parametrize("case", range(len(CASES)))
@pytest.mark.parametrize("out", ["bf16", "fp32"])
def test_attention(bd, case, out):
    lens, rows, shares, page, Hk, G, d, block = CASES[case]
    c = tree(case, lens, shares, page=page, Hk=Hk, d=d, layers=2)
    off, n = cu.offsets(rows), len(lens)
    T = int(off[-1]) + 2
    q = torch.from_numpy(np.random.default_rng(case).standard_normal((T, Hk * G, d))).bfloat16().cuda()
    cache = cu.to_device(bd, c)
    o = torch.full((T, Hk * G, d), 7.0, dtype=torch.float32 if out == "fp32" else torch.bfloat16, device="cuda")
    lse = torch.full((Hk * G, T), 9.0, device="cuda")
    bd.bdlm_cache_attn_shared_fwd(cache, q, dev(off), block, dev(plan_of(n, shares, page)), layer=1, out=o, lse=lse, check=True)
    ref = co.attention(c, 1, q.double().cpu().numpy(), off, block, d ** -0.5)
    keep = int(off[-1])
    cu.check_attention(o[:keep], lse[:, :keep], tuple(x[:, :keep] if x.shape[0] == Hk * G and x.ndim == 2 else x[:keep] for x in ref), f"case {case}")
    assert torch.all(o[keep:] == 7.0) and torch.all(lse[:, keep:] == 9.0)
    found = bd.bdlm_cache_prefixes(cache, dev(off), check=True)  # what the plan finds gives the same
    o2, lse2 = bd.bdlm_cache_attn_shared_fwd(cache, q, dev(off), block, found, layer=1, out=torch.zeros_like(o), check=True)
    cu.check_attention(o2[:keep], lse2[:, :keep], tuple(x[:, :keep] if x.shape[0] == Hk * G and x.ndim == 2 else x[:keep] for x in ref), f"case {case}, found")


@pytest.mark.parametrize("seed", range(12))
def test_random_trees(bd, seed):
    """Prompts with candidates, found runs, ragged everything; and the positions given (q_pos) as the decoder does."""
    rng = np.random.default_rng(100 + seed)
    page, Hk, G, d = int(rng.choice([16, 32, 64, 128])), int(rng.integers(1, 4)), int(rng.choice([1, 2, 3, 4, 7])), int(rng.choice([64, 128]))
    lens, rows, shares = [], [], []
    for _ in range(int(rng.integers(1, 6))):
        prefix, kids = int(rng.integers(1, 1500)), int(rng.integers(1, 9))
        if kids > 1 and prefix >= page:
            shares.append((len(lens), len(lens) + kids, prefix // page))
        for _ in range(kids):
            r = int(rng.integers(0, 40))
            lens.append(prefix + r + int(rng.integers(0, 100)))
            rows.append(r)
    if sum(rows) == 0:
        rows[0], lens[0] = 1, lens[0] + 1
    block = int(rng.choice([1, 8, 32, 45]))
    c = tree(seed, lens, shares, page=page, Hk=Hk, d=d)
    off = cu.offsets(rows)
    q = torch.from_numpy(rng.standard_normal((int(off[-1]), Hk * G, d))).bfloat16().cuda()
    cache = cu.to_device(bd, c)
    runs = bd.bdlm_cache_prefixes(cache, dev(off), check=True)
    ref = co.attention(c, 0, q.double().cpu().numpy(), off, block, d ** -0.5)
    cu.check_attention(*bd.bdlm_cache_attn_shared_fwd(cache, q, dev(off), block, runs, check=True), ref, f"seed {seed}")
    pos = np.asarray(lens) - rows
    runs = bd.bdlm_cache_prefixes(cache, dev(off), q_pos=dev(pos), check=True)
    cu.check_attention(*bd.bdlm_cache_attn_shared_fwd(cache, q, dev(off), block, runs, q_pos=dev(pos), check=True), ref, f"seed {seed}, positions")


def test_keys_beyond_the_cache(bd):
    """Rows whose own keys are not in the cache (q_pos): a sequence may hold nothing but what it shares, or nothing at all."""
    page, Hk, G, d = 16, 2, 2, 64
    lens, rows, shares = [64, 64, 80, 0], [3, 3, 3, 2], [(0, 3, 4)]
    c = tree(1, lens, shares, page=page, Hk=Hk, d=d)
    off, pos = cu.offsets(rows), [64, 70, 80, 5]
    q = torch.randn(int(off[-1]), Hk * G, d, device="cuda").bfloat16()
    cache = cu.to_device(bd, c)
    ref = co.attention(c, 0, q.double().cpu().numpy(), off, 4, d ** -0.5, q_pos=pos)
    for plan in (dev(plan_of(4, shares, page)), bd.bdlm_cache_prefixes(cache, dev(off), q_pos=dev(pos), check=True)):
        cu.check_attention(*bd.bdlm_cache_attn_shared_fwd(cache, q, dev(off), 4, plan, q_pos=dev(pos), check=True), ref)


def test_no_number_in_one_branch(bd):
    """NaN in a candidate's own page reaches its rows alone; NaN in a shared page those of the run."""
    page, Hk, G, d = 16, 1, 2, 64
    lens, rows, shares = [70, 75, 80, 60], [2, 2, 2, 2], [(0, 3, 3)]
    for where in ((1, 4), (0, 1), (3, 0)):
        c = tree(2, lens, shares, page=page, Hk=Hk, d=d)
        c["v"][0, c["table"][where], 0, 2, 5] = 127
        off = cu.offsets(rows)
        q = torch.randn(8, Hk * G, d, device="cuda").bfloat16()
        cache = cu.to_device(bd, c)
        ref = co.attention(c, 0, q.double().cpu().numpy(), off, 1, d ** -0.5)
        cu.check_attention(*bd.bdlm_cache_attn_shared_fwd(cache, q, dev(off), 1, dev(plan_of(4, shares, page)), check=True), ref, str(where))


@pytest.mark.parametrize("d,page,G,rows,block", [(64, 16, 1, 8, 1), (128, 16, 1, 8, 3), (64, 32, 2, 4, 2), (128, 64, 4, 2, 1), (64, 128, 8, 1, 1),
                                                 (128, 32, 3, 2, 1), (128, 16, 5, 1, 1), (64, 16, 1, 7, 4)])
def test_few_rows(bd, d, page, G, rows, block):
    """Up to eight flat rows, with blocks that end within 16 keys: rows see different numbers of them, and NaN among the values
    that only the later rows see reaches those alone. Rows of q far from 1, and pages of unlike magnitude."""
    Hk, prefix = 2, 1792
    own = [rows, rows + 1, rows + 5, 15 + rows, 16 + rows, 37, 128 + rows, 300, 2048]
    lens, n = [prefix + x for x in own], len(own)
    shares = [(0, n, prefix // page)]
    c = tree(page + G, lens, shares, page=page, Hk=Hk, d=d, page_spread=3.0)
    off = cu.offsets([rows] * n)
    rng = np.random.default_rng(rows)
    q = torch.from_numpy(rng.standard_normal((int(off[-1]), Hk * G, d)) * np.exp2(rng.choice([-70, -8, 0, 0, 0, 3, 20], (int(off[-1]), Hk * G, 1))))
    q = q.bfloat16().cuda()
    for marks in (0, 1):
        if marks:
            for s in range(n):  # the last row's own key, and the one in the middle of the rows
                for back, col in ((1, 3), (rows // 2 + 1, d - 1)):
                    at = lens[s] - back
                    c["v"][0, c["table"][s, at // page], s % 2, at % page, col] = 127
        cache = cu.to_device(bd, c)
        ref = co.attention(c, 0, q.double().cpu().numpy(), off, block, d ** -0.5)
        runs = bd.bdlm_cache_prefixes(cache, dev(off), check=True)
        for plan in (runs, dev(plan_of(n, [], page))):
            o, lse = torch.empty(q.shape, dtype=torch.float32, device="cuda"), torch.empty((Hk * G, q.shape[0]), device="cuda")
            bd.bdlm_cache_attn_shared_fwd(cache, q, dev(off), block, plan, out=o, lse=lse, check=True)
            # An o is at most A, so where the scores' own error of 2^-15 S1 allows a difference of 2 A and more, as it does from
            # S1 = 2^15 on, the bound says nothing of o; the weights of scores from 2^23 on, which fp32 holds to whole
            # octaves, may be anything.
            void = 2.0 ** -14 * ref[3].T >= 2
            o[torch.from_numpy(void).cuda()] = torch.from_numpy(ref[0][void]).float().cuda()
            cu.check_attention(o, lse, ref, f"NaN {marks}")


@pytest.mark.parametrize("d,page", [(64, 16), (128, 128)])
def test_few_rows_of_many_sequences(bd, d, page):
    """Enough sequences that own keys up to 4096 count as few; one has more."""
    n, Hk, prefix = 33, 8, 2048
    own = [1 + 7 * s for s in range(n)]
    own[3], own[7], own[8], own[20], own[32] = 2049, 4095, 4096, 4097, 3000
    lens = [prefix + x for x in own]
    c = tree(d, lens, [(0, n, prefix // page)], page=page, Hk=Hk, d=d)
    off = cu.offsets([1] * n)
    q = torch.from_numpy(np.random.default_rng(d).standard_normal((n, Hk, d))).bfloat16().cuda()
    cache = cu.to_device(bd, c)
    ref = co.attention(c, 0, q.double().cpu().numpy(), off, 1, d ** -0.5)
    runs = bd.bdlm_cache_prefixes(cache, dev(off), check=True)
    assert runs[2].tolist() == [prefix] * n
    cu.check_attention(*bd.bdlm_cache_attn_shared_fwd(cache, q, dev(off), 1, runs, check=True), ref)


BAD_PLANS = [
    [[0, 0, 0], [3, 3, 3], [32, 32, 16]],   # not the same
    [[0, 0, 2], [3, 3, 3], [32, 32, 32]],
    [[0, 0, 0], [3, 2, 3], [32, 32, 32]],
    [[0, 0, 0], [4, 4, 4], [32, 32, 32]],   # beyond the sequences
    [[-1, -1, -1], [3, 3, 3], [32, 32, 32]],
    [[0, 0, 0], [3, 3, 3], [24, 24, 24]],   # no whole pages
    [[0, 0, 0], [3, 3, 3], [48, 48, 48]],   # more than the rows see
    [[0, 0, 0], [3, 3, 3], [-16, -16, -16]],
    [[0, 1, 1], [1, 1, 3], [0, 0, 0]],
    [[0, 1, 2], [1, 2, 2], [0, 0, 0]],
    [[2 ** 31 - 1] * 3, [-2 ** 31] * 3, [2 ** 31 - 16] * 3],
]


@pytest.mark.parametrize("plan", BAD_PLANS, ids=str)
def test_malformed_plans(bd, plan):
    c = tree(3, [40, 45, 44], [(0, 3, 2)], page=16, Hk=1, d=64)
    cache = cu.to_device(bd, c)
    q = torch.randn(3, 2, 64, device="cuda").bfloat16()
    o, lse = torch.full((3, 2, 64), 5.0, device="cuda").bfloat16(), torch.full((2, 3), 5.0, device="cuda")
    with pytest.raises(bd.BDLMError):
        bd.bdlm_cache_attn_shared_fwd(cache, q, dev([0, 1, 2, 3]), 1, dev(plan), out=o, lse=lse, check=True)
    assert torch.all(o == 5.0) and torch.all(lse == 5.0)


def test_malformed_offsets_and_pages(bd):
    c = tree(3, [40, 45, 44], [(0, 3, 2)], page=16, Hk=1, d=64)
    cache = cu.to_device(bd, c)
    plan = dev(plan_of(3, [(0, 3, 2)], 16))
    q = torch.randn(3, 2, 64, device="cuda").bfloat16()
    for off in ([0, 1, 2, 4], [0, 2, 1, 3], [1, 1, 2, 3]):
        with pytest.raises(bd.BDLMError):
            bd.bdlm_cache_attn_shared_fwd(cache, q, dev(off), 1, plan, check=True)
    cache.table[1, 2] = 10 ** 6  # a page of its own outside the pool: its rows alone are NaN
    ws = torch.zeros(bd.bdlm_cache_attn_shared_fwd_workspace_bytes(3, 2, 1, 64, 3), dtype=torch.uint8, device="cuda")
    o, _ = bd.bdlm_cache_attn_shared_fwd(cache, q, dev([0, 1, 2, 3]), 1, plan, workspace=ws)
    assert bd.bdlm_read_error(ws) == 6
    assert torch.isnan(o[1]).all() and torch.isfinite(o[0]).all() and torch.isfinite(o[2]).all()


def test_captured_and_on_another_stream(bd):
    lens, rows, shares = [700, 720, 800, 90], [16, 16, 16, 16], [(0, 3, 10)]
    c = tree(9, lens, shares, page=64, Hk=2, d=128)
    cache, off = cu.to_device(bd, c), dev(cu.offsets(rows))
    q = torch.randn(64, 8, 128, device="cuda").bfloat16()
    runs = bd.bdlm_cache_prefixes(cache, off)
    want = bd.bdlm_cache_attn_shared_fwd(cache, q, off, 16, runs)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    plan = bd.bdlm_cache_prefixes(cache, off, stream=side)
    got = bd.bdlm_cache_attn_shared_fwd(cache, q, off, 16, plan, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(plan, runs) and torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    graph, o, lse = torch.cuda.CUDAGraph(), torch.empty_like(want[0]), torch.empty_like(want[1])
    with torch.cuda.graph(graph):
        plan = bd.bdlm_cache_prefixes(cache, off, out=plan)
        bd.bdlm_cache_attn_shared_fwd(cache, q, off, 16, plan, out=o, lse=lse)
    cache.table[2, 4:10] = cache.table[2, 4:10].flip(0)  # another tree, other queries
    q.copy_(torch.randn(64, 8, 128, device="cuda").bfloat16())
    graph.replay()
    runs = bd.bdlm_cache_prefixes(cache, off)
    want = bd.bdlm_cache_attn_shared_fwd(cache, q, off, 16, runs)
    assert torch.equal(plan, runs) and torch.equal(o, want[0]) and torch.equal(lse, want[1])


def test_no_rows(bd):
    cache = bd.PageCache.empty(1, 4, 16, 1, 64, 2, 3)
    off = dev([0, 0, 0])
    runs = bd.bdlm_cache_prefixes(cache, off, check=True)
    o, lse = bd.bdlm_cache_attn_shared_fwd(cache, torch.zeros((0, 2, 64), device="cuda").bfloat16(), off, 1, runs, check=True)
    assert o.shape == (0, 2, 64) and lse.shape == (2, 0) and runs.tolist() == [[0, 1], [1, 2], [0, 0]]


def test_refusals(bd):
    cache = bd.PageCache.empty(1, 4, 16, 1, 64, 2, 3)
    q, off = torch.zeros((2, 2, 64), device="cuda").bfloat16(), dev([0, 1, 2])
    for runs in (dev([[0, 1], [1, 2]]), dev([[0, 1], [1, 2], [0, 0]]).long(), dev([[0, 1], [1, 2], [0, 0]]).cpu(), None,
                 dev([[0, 1, 0], [1, 2, 0]]).t()):
        with pytest.raises(ValueError):
            bd.bdlm_cache_attn_shared_fwd(cache, q, off, 1, runs)
    with pytest.raises(ValueError):
        bd.bdlm_cache_prefixes(cache, off[:2])
    with pytest.raises(ValueError):
        bd.bdlm_cache_prefixes(cache, off, out=dev([0, 1]))
