"""Sampling where the three cuts meet: top-p goes by what the first k tokens weigh together, also those that min-p drops
afterwards. Tokens have to equal the float64 oracle's; log-probabilities have test_gpu_sample's bound."""
import math

import numpy as np
import pytest
import torch

from test_gpu_sample import DTYPES, bd, check  # noqa: F401  (bd is a fixture)

pytestmark = pytest.mark.gpu

HOW = [(k, p, m) for k in (200, 300, 500, 1000, 2000, 0.25, 0.5) for p in (0.3, 0.5, 0.8, 0.9) for m in (0.01, 0.05, 0.1, 0.2)]


def flat(seed, rows, vocab, dtype, heads):
    """Rows whose tail weighs as much as what stands out of it, or more; every other one with `heads` tokens at 6."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((rows, vocab))
    for r in range(0, rows, 2):
        x[r, rng.choice(vocab, heads, replace=False)] = 6.0
    return torch.from_numpy(x).to(dtype).cuda()


def columns(rows, vocab, seed):
    rng = np.random.default_rng(seed)
    how = [HOW[i] for i in rng.permutation(len(HOW))]
    how = [how[r % len(how)] for r in range(rows)]
    t = lambda v, dt: torch.tensor(v, dtype=dt, device="cuda")
    return {"top_k": t([k if k > 1 else int(k * vocab) for k, _, _ in how], torch.int32), "top_p": t([p for _, p, _ in how], torch.float32),
            "min_p": t([m for _, _, m in how], torch.float32)}


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("vocab,rows", [(32768, 160), (131072, 24), (131072, 9), (5003, 224)])
def test_top_k_weighs_what_min_p_drops(bd, dtype, vocab, rows):
    """Rows of one, two, four and eight CTAs, of more and of fewer tokens than a list holds."""
    x, how = flat(vocab + rows, rows, vocab, DTYPES[dtype], 20), columns(rows, vocab, rows)
    u = torch.rand(rows, generator=torch.Generator("cuda").manual_seed(rows), device="cuda")
    check(bd, x, u, **how)
    check(bd, x, u, temperature=0.8, **how)


@pytest.mark.parametrize("dtype", DTYPES)
def test_all_cuts_alone_and_among_others(bd, dtype):
    """A row's token is the same however many CTAs take it."""
    vocab, rows = 32768, 160
    x, how = flat(7, rows, vocab, DTYPES[dtype], 20), columns(rows, vocab, 1)
    u = torch.rand(rows, generator=torch.Generator("cuda").manual_seed(3), device="cuda")
    token, _ = bd.bdlm_sample(x, u, **how)
    for r in range(0, rows, 5):
        one, _ = bd.bdlm_sample(x[r:r + 1], u[r:r + 1], **{name: t[r:r + 1] for name, t in how.items()})
        assert one.item() == token[r].item(), r


@pytest.mark.parametrize("dtype", DTYPES)
def test_all_cuts_over_few_tokens(bd, dtype):
    """Most tokens are masked: the list has all that are left, fewer than k."""
    vocab, rows = 20000, 32
    x = flat(3, rows, vocab, DTYPES[dtype], 20)
    rng = np.random.default_rng(4)
    for r, left in enumerate(np.repeat([1, 2, 31, 32, 33, 127, 128, 500], 4)):
        gone = torch.ones(vocab, dtype=torch.bool)
        gone[torch.from_numpy(rng.choice(vocab, left, replace=False))] = False
        x[r, gone.cuda()] = float("-inf")
    u = torch.rand(rows, generator=torch.Generator("cuda").manual_seed(5), device="cuda")
    for how in (dict(top_k=2000, top_p=0.5, min_p=0.05), dict(top_k=100, top_p=0.9, min_p=0.2), dict(top_k=400, top_p=0.7, min_p=0.001)):
        check(bd, x, u, **how)


@pytest.mark.parametrize("rows", [24, 9])
def test_border_between_light_tokens(bd, rows):
    """Rows of four and eight CTAs without cuts, whose counted values decide. The first CTA has tokens of 0.47 units of 2^-44 each, which
    weigh nothing, and two of 59844 units behind them: a draw that falls between those two goes by exact weights alone."""
    vocab = 131072
    part = vocab // (4 if rows > 19 else 8)
    x = torch.zeros((rows, vocab), dtype=torch.bfloat16, device="cuda")
    x[:, :part - 2] = -31.25
    x[:, part - 2:part] = -19.5
    units = (vocab - part) * 2.0 ** 44
    at = torch.tensor([1000, 30000, 52000, 59000, 61000, 63000, 67000, 75000, 100000] * 3, dtype=torch.float64)[:rows]
    check(bd, x, (at / units).float().cuda())


@pytest.mark.parametrize("dtype", ["fp16", "fp32"])
def test_top_p_far_from_where_quick_sums_put_it(bd, dtype):
    """200 heavy tokens whose bins' sums are off by 4e-6 of themselves, more than thousands of the light ones weigh, and top-p
    cuts among those: the cut is found in a few tens of passes (of about 15 us), not one token at a time."""
    vocab, rows = 131072, 3
    rng = np.random.default_rng(8)
    x = rng.uniform(-1, 1, (rows, vocab))
    for r in range(rows):
        some = rng.choice(vocab, 201, replace=False)
        x[r, some] = 15 - math.log(2) / 8
        x[r, some[0]] = 15
    x = torch.from_numpy(x).to(DTYPES[dtype]).cuda()
    w = torch.exp(x.double() - x.double().amax(1, keepdim=True))
    top = x.double() > 5
    heavy, light = (w * top).sum(1), (w * ~top).sum(1)
    p = ((heavy + light * torch.tensor([0.1, 0.5, 0.9], device="cuda", dtype=torch.float64)) / (heavy + light)).float()
    for u in (1.0, 0.9999, 0.99995, 0.3):
        check(bd, x, torch.full((rows,), u, device="cuda"), top_p=p)
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    u = torch.full((rows,), 0.5, device="cuda")
    start.record()
    for _ in range(10):
        bd.bdlm_sample(x, u, top_p=p)
    end.record()
    end.synchronize()
    assert start.elapsed_time(end) / 10 < 5.0  # ms
