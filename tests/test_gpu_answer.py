"""Prompts, candidates, shared attention, sampling and unmasking together, as decode.BlockDecoder runs them, against the
float64 oracles; from eager calls and from captured graphs."""
import numpy as np
import pytest
import torch

from oracle import answer_oracle as ao
from oracle import cache_oracle as co

import cache_util as cu

pytestmark = pytest.mark.gpu
MASK = 499


@pytest.fixture(scope="module")
def bd():
    import block_diffusion_lm_bdlm_gb300 as m

    m.load_library()
    return m


def dev(x, dtype=torch.int32):
    return torch.as_tensor(np.asarray(x)).to("cuda", dtype)


def start(bd, page, Hk, d, prompts, kids, block, share):
    """Prompts of ragged lengths in sequences 0 .., their candidates side by side behind them."""
    from block_diffusion_lm_bdlm_gb300.decode import BlockDecoder

    n = len(prompts) * (1 + kids)
    need = sum(co.pages_of(p, page) + kids * (1 + 2 * co.pages_of(block, page)) for p in prompts) + 4
    cache = bd.PageCache.empty(1, need, page, Hk, d, n, co.pages_of(max(prompts) + 3 * block, page))
    cache.k.view(torch.uint8).fill_(127)  # NaN wherever nothing is written
    cache.v.view(torch.uint8).fill_(127)
    dec = BlockDecoder(cache, block, share=share)
    gen = torch.Generator("cuda").manual_seed(1)
    dec.begin(dev(prompts + [0] * (n - len(prompts))), check=True)
    T = sum(prompts)
    q, k, v = (torch.randn(T, h, d, device="cuda", generator=gen).bfloat16() for h in (2 * Hk, Hk, Hk))
    dec.attend(0, q, k, v, check=True)
    parents = [i for i in range(len(prompts)) for _ in range(kids)]
    dec.branch(dev(parents), dev(range(len(prompts), n)), check=True)
    dec.end(dev(range(len(prompts))))
    return dec, gen, n


@pytest.mark.parametrize("page,Hk,d,prompts,kids,block", [(16, 1, 64, [3000, 90, 1700], 5, 8), (64, 2, 128, [2500], 9, 4),
                                                          (128, 2, 64, [40, 700], 2, 32)])
def test_blocks(bd, page, Hk, d, prompts, kids, block):
    """Two blocks of every candidate, step by step: attention, drawn tokens and kept rows are the oracles'."""
    dec, gen, n = start(bd, page, Hk, d, prompts, kids, block, True)
    cache, vocab = dec.cache, 500
    for _ in range(2):
        rows = [0] * len(prompts) + [block] * (n - len(prompts))
        off = dec.begin(dev(rows), check=True).cpu().numpy()
        T = int(off[-1])
        tokens, left = torch.full((T,), MASK, dtype=torch.int32, device="cuda"), None
        for step in range(3):
            q, k, v = (torch.randn(T, h, d, device="cuda", generator=gen).bfloat16() for h in (2 * Hk, Hk, Hk))
            o, lse = dec.attend(0, q, k, v, check=True)
            ref = co.attention(cu.to_host(cache), 0, q.double().cpu().numpy(), off, block, d ** -0.5)
            cu.check_attention(o, lse, ref, f"step {step}")
            logits = (4 * torch.randn(T, vocab, device="cuda", generator=gen)).bfloat16()
            logits[:, MASK] = float("-inf")
            u, was = torch.rand(T, device="cuda", generator=gen), tokens.cpu().numpy()
            n_min, thr = max(1, block // 4), -0.7
            left = dec.choose(tokens, logits, u, MASK, temperature=0.9, top_k=50, top_p=0.9, n_min=n_min, threshold=thr, check=True)
            x, uh = logits.double().cpu().numpy(), u.double().cpu().numpy()
            f32 = lambda y: float(np.float32(y))
            drawn = [ao.sample_row(x[i], uh[i], f32(0.9), 50, f32(0.9)) if was[i] == MASK else (-1, 0.0) for i in range(T)]
            want, wleft = ao.unmask(was, [t for t, _ in drawn], np.float32([p for _, p in drawn]), off, MASK, [n_min] * n, [np.float32(thr)] * n)
            assert np.array_equal(tokens.cpu().numpy(), want) and np.array_equal(left.cpu().numpy(), wleft)
        dec.choose(tokens, logits, u, MASK, n_min=block, check=True)
        assert not bool((tokens == MASK).any())


def test_sharing_changes_sums_only(bd):
    """Each call of a life with candidates, ended ones, a rewound block: with and without sharing the same rows."""
    got = []
    for share in (False, True):
        dec, gen, n = start(bd, 16, 2, 64, [1900, 64], 4, 8, share)
        out = []

        def step(T):
            q, k, v = (torch.randn(T, h, 64, device="cuda", generator=gen).bfloat16() for h in (4, 2, 2))
            out.append(dec.attend(0, q, k, v, check=False))

        dec.begin(dev([0, 0] + [8] * 8), check=True)
        step(64)
        dec.end(dev([3, 6]))  # in the middle of the block: their rows see nothing, the others go on
        step(64)
        dec.rewind()
        dec.begin(dev([0, 0, 8, 0, 8, 1, 0, 3, 8, 8]), check=True)
        step(36)
        dec.branch(dev([2]), dev([3]), check=True)
        dec.begin(dev([0, 0, 8, 8, 8, 8, 0, 8, 8, 8]), check=True)
        step(56)
        got.append(out)
    for (o, lse), (o1, lse1) in zip(*got):
        assert torch.equal(torch.isneginf(lse), torch.isneginf(lse1))
        seen = ~torch.isneginf(lse)
        assert torch.allclose(lse[seen], lse1[seen], rtol=0, atol=2e-3) and torch.allclose(o.float(), o1.float(), rtol=0, atol=2e-2)


def test_captured_step(bd):
    """A denoising step (attention, drawing, keeping) replayed on new queries, logits and numbers."""
    dec, gen, n = start(bd, 16, 1, 64, [2100], 6, 4, True)
    T, vocab = 24, 300
    dec.begin(dev([0] + [4] * 6), check=True)
    q, k, v = (torch.randn(T, h, 64, device="cuda", generator=gen).bfloat16() for h in (2, 1, 1))
    logits, u = torch.randn(T, vocab, device="cuda", generator=gen), torch.rand(T, device="cuda", generator=gen)
    tokens = torch.full((T,), MASK, dtype=torch.int32, device="cuda")
    o, lse = torch.empty_like(q), torch.empty(2, T, device="cuda")

    def step():
        dec.attend(0, q, k, v, out=o, lse=lse)
        return dec.choose(tokens, logits, u, MASK, top_p=0.8)

    step()
    tokens.fill_(MASK)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        left = step()
    for _ in range(3):
        for x in (q, k, v, logits):
            x.copy_(torch.randn(x.shape, device="cuda", generator=gen))
        u.copy_(torch.rand(T, device="cuda", generator=gen))
        was = tokens.clone()
        graph.replay()
        got = o.clone(), lse.clone(), tokens.clone(), left.clone()
        tokens.copy_(was)
        again = step()
        assert torch.equal(got[0], o) and torch.equal(got[1], lse) and torch.equal(got[2], tokens) and torch.equal(got[3], again)


def test_calls_of_several_threads(bd):
    """Calls of unlike sizes from four threads at once, each on a stream of its own, give what they give one after the other."""
    from concurrent.futures import ThreadPoolExecutor

    gen = torch.Generator("cuda").manual_seed(9)
    jobs = []
    for vocab, dtype, n in ((100, torch.float32, 5), (262144, torch.float32, 12000), (32001, torch.bfloat16, 40), (131072, torch.float16, 16384)):
        logits, u = (2 * torch.randn(3, vocab, device="cuda", generator=gen)).to(dtype), torch.rand(3, device="cuda", generator=gen)
        cache = bd.PageCache.empty(1, 4, 16, 1, 64, n, 2)
        cache.lens.fill_(17)  # all in the same pages: runs of 256
        jobs.append((logits, u, cache, torch.arange(n + 1, dtype=torch.int32, device="cuda"), torch.cuda.Stream()))

    def work(job, times):
        logits, u, cache, cu_rows, stream = job
        got = []
        for _ in range(times):
            token, lp = bd.bdlm_sample(logits, u, top_p=0.9, stream=stream)
            got.append((token, lp, bd.bdlm_cache_prefixes(cache, cu_rows, stream=stream)))
        stream.synchronize()
        return got

    torch.cuda.synchronize()
    want = [work(job, 1)[0] for job in jobs]
    with ThreadPoolExecutor(len(jobs)) as pool:
        for ref, got in zip(want, pool.map(lambda job: work(job, 50), jobs)):
            assert all(torch.equal(x, y) for one in got for x, y in zip(ref, one))
