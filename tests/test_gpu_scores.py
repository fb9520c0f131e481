"""Scores up to 2^22, where fp32 holds them to a quarter: what they weigh may be off, but o stays a mean of the values.

A weight enters as fp16 (2^-11 of it, above and below the fraction bar) or as two such terms, sums are fp32 (2^-12), and o is
rounded to its type: each entry lies between the least and the largest value that the row sees in that column, give or take
2^-10 + 2^-12 + u of the largest magnitude."""
import numpy as np
import pytest
import torch

from oracle import cache_oracle as co

import cache_util as cu
from test_gpu_shared import bd, dev, plan_of, tree  # noqa: F401  (bd is a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32], ids=str)
@pytest.mark.parametrize("d,page,G,rows,own", [(64, 16, 1, 8, 40), (128, 64, 4, 2, 300), (128, 128, 2, 40, 700), (64, 32, 8, 70, 100), (128, 16, 1, 1, 2500)])
def test_large_scores_keep_o_within_the_values(bd, d, page, G, rows, own, out):
    Hk, n = 2, 5
    prefix = 1280
    lens = [prefix + own + 3 * s for s in range(n)]
    shares = [(0, n, prefix // page)]
    c = tree(d + rows, lens, shares, page=page, Hk=Hk, d=d, page_spread=2.0)
    off = cu.offsets([rows] * n)
    T = int(off[-1])
    rng = np.random.default_rng(rows)
    q = rng.standard_normal((T, Hk * G, d))
    lo, hi = np.empty((2, T, Hk * G, d))
    for s in range(n):
        ids = c["table"][s, :co.pages_of(lens[s], page)]
        for h in range(Hk):
            k, v = ((co.VALUES[c[x][0, ids, h]] * c[x + "s"][0, ids, h][:, None, None]).reshape(-1, d)[:lens[s]] for x in "kv")
            for i in range(off[s], off[s + 1]):
                end = lens[s] - (off[s + 1] - 1 - i)  # block 1
                for g in range(h * G, h * G + G):
                    top = np.abs(k[:end] @ q[i, g]).max() * d ** -0.5
                    # largest score in (2^(e-1), 2^e): a sixteenth to spare for the rounding of q to bf16
                    q[i, g] *= 2.0 ** int(rng.integers(15, 23)) * (15 / 16) / top * rng.choice([1.0, 0.53])
                    lo[i, g], hi[i, g] = v[:end].min(0), v[:end].max(0)
    q = torch.from_numpy(q).bfloat16().cuda()
    cache = cu.to_device(bd, c)
    u = torch.finfo(out).eps / 2
    slack = (2.0 ** -10 + 2.0 ** -12 + u) * np.maximum(np.abs(lo), np.abs(hi))
    for call in ((bd.bdlm_cache_attn_fwd,), (bd.bdlm_cache_attn_shared_fwd, dev(plan_of(n, shares, page))),
                 (bd.bdlm_cache_attn_shared_fwd, dev(plan_of(n, [], page)))):
        o, lse = call[0](cache, q, dev(off), 1, *call[1:], out=torch.empty(q.shape, dtype=out, device="cuda"), check=True)
        o = o.double().cpu().numpy()
        assert np.all(np.isfinite(o)) and torch.isfinite(lse).all()
        assert np.all(o >= lo - slack) and np.all(o <= hi + slack), float(np.maximum(lo - o, o - hi).max())
