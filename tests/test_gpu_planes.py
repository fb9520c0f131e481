"""Partial results of rows that are read together, in calls with many more rows than those: their places go by sequence.
(test_gpu_shared holds the bounds' reasons.)"""
import numpy as np
import pytest
import torch

from oracle import cache_oracle as co

import cache_util as cu
from test_gpu_shared import bd, dev, plan_of, tree  # noqa: F401  (bd is a fixture)

pytestmark = pytest.mark.gpu

# lens, rows, shares, page, Hk, G, d, block: more than 128 flat rows for each sequence in all
CASES = [
    ([700] + [2100] * 6, [640] + [1, 2, 1, 1, 2, 1], [(1, 7, 32)], 64, 2, 4, 64, 32),               # few rows behind a prompt
    ([2600] * 5 + [900] + [2200, 2300, 2200], [9, 20, 7, 16, 9, 800, 3, 1, 5], [(0, 5, 40), (6, 9, 16)], 64, 1, 4, 128, 16),
    ([1500, 1600, 1400] * 4 + [1100], [16] * 12 + [1000], [(0, 12, 80)], 16, 2, 3, 64, 20),           # cut units of a run
    ([500, 40, 40, 900], [400, 0, 0, 300], [], 16, 2, 2, 64, 32),                                     # no run at all
    ([3000, 3000, 700, 3000], [5, 0, 600, 7], [(0, 2, 100)], 16, 1, 7, 128, 3),
]


@pytest.mark.parametrize("case", range(len(CASES)))
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32], ids=str)
def test_rows_behind_prompts(bd, case, out):
    lens, rows, shares, page, Hk, G, d, block = CASES[case]
    c = tree(40 + case, lens, shares, page=page, Hk=Hk, d=d)
    off, n = cu.offsets(rows), len(lens)
    T = int(off[-1])
    assert T * G > 128 * n
    q = torch.from_numpy(np.random.default_rng(case).standard_normal((T, Hk * G, d))).bfloat16().cuda()
    cache = cu.to_device(bd, c)
    ref = co.attention(c, 0, q.double().cpu().numpy(), off, block, d ** -0.5)
    need = bd.bdlm_cache_attn_shared_fwd_workspace_bytes(T, Hk * G, Hk, d, n)
    for plan in (dev(plan_of(n, shares, page)), bd.bdlm_cache_prefixes(cache, dev(off), check=True)):
        ws = torch.full((need + 8192,), 255, dtype=torch.uint8, device="cuda")
        o, lse = torch.empty(q.shape, dtype=out, device="cuda"), torch.empty((Hk * G, T), device="cuda")
        bd.bdlm_cache_attn_shared_fwd(cache, q, dev(off), block, plan, out=o, lse=lse, workspace=ws[:need], check=True)
        cu.check_attention(o, lse, ref, f"case {case}")
        assert torch.all(ws[need:] == 255)


@pytest.mark.parametrize("seed", range(10))
def test_random_trees_with_prompts(bd, seed):
    rng = np.random.default_rng(300 + seed)
    page, Hk, G, d = int(rng.choice([16, 64])), int(rng.integers(1, 3)), int(rng.choice([2, 4, 7])), int(rng.choice([64, 128]))
    lens, rows, shares = [], [], []
    for _ in range(int(rng.integers(2, 5))):
        if rng.random() < 0.5:
            r = int(rng.integers(500, 1200))
            lens.append(r + int(rng.integers(0, 200)))
            rows.append(r)
        prefix, kids = int(rng.integers(2000, 4000)), int(rng.integers(3, 9))
        shares.append((len(lens), len(lens) + kids, prefix // page))
        for _ in range(kids):
            r = int(rng.integers(0, 1 + int(rng.choice([2, 12]))))
            lens.append(prefix + r + int(rng.integers(0, 300)))
            rows.append(r)
    rows.append(128 * len(rows) // G + 300)
    lens.append(rows[-1])
    c = tree(seed, lens, shares, page=page, Hk=Hk, d=d)
    off = cu.offsets(rows)
    q = torch.from_numpy(rng.standard_normal((int(off[-1]), Hk * G, d))).bfloat16().cuda()
    cache = cu.to_device(bd, c)
    ref = co.attention(c, 0, q.double().cpu().numpy(), off, 32, d ** -0.5)
    for plan in (bd.bdlm_cache_prefixes(cache, dev(off), check=True), dev(plan_of(len(rows), shares, page))):
        cu.check_attention(*bd.bdlm_cache_attn_shared_fwd(cache, q, dev(off), 32, plan, check=True), ref, f"seed {seed}")
