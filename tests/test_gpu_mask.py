"""The mask is a token of the vocabulary: a row that draws it is still masked, and a denoising step does not draw it."""
import math

import numpy as np
import pytest
import torch

from oracle import answer_oracle as ao

from test_gpu_sample import bd  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu


def dev(x, dtype=torch.int32):
    return torch.as_tensor(np.asarray(x)).to("cuda", dtype)


@pytest.mark.parametrize("rows", [[1], [32] * 16, [0, 5, 1, 0, 33, 257, 7], [1024, 1025, 2]], ids=str)
@pytest.mark.parametrize("share", [0.2, 1.0])
@pytest.mark.parametrize("mask", [77, 0])
def test_a_drawn_mask_is_no_token(bd, rows, share, mask):
    """`left` counts the rows whose token is the mask afterwards, and the surest others take the place of those that drew it."""
    rng = np.random.default_rng(len(rows))
    T, n = sum(rows), len(rows)
    off = np.concatenate([[0], np.cumsum(rows)])
    tokens = np.where(rng.random(T) < 0.7, mask, 5)
    sampled = np.where(rng.random(T) < share, mask, rng.integers(100, 200, T))
    lp = (-np.round(rng.random(T) * 8) / 8).astype(np.float32)
    lp[sampled == mask] = 0.0  # the surest
    for k, thr in ((0, -0.25), (4, math.nan), (1000, -0.5)):
        want, left = ao.unmask(tokens, sampled, lp, off, mask, [k] * n, [thr] * n)
        assert left.tolist() == [int((want[a:b] == mask).sum()) for a, b in zip(off, off[1:])]
        t = dev(tokens)
        for out in (torch.empty_like(t), t):
            got, gl = bd.bdlm_unmask(t, dev(sampled), dev(lp, torch.float32), dev(off), mask, n_min=k, threshold=thr, out=out, check=True)
            assert np.array_equal(got.cpu().numpy(), want) and np.array_equal(gl.cpu().numpy(), left)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32], ids=str)
@pytest.mark.parametrize("vocab,rows,pad", [(1, 2, 0), (2, 3, 1), (40, 9, 0), (4099, 160, 5), (131072, 5, 0), (131072, 40, 3)])
@pytest.mark.parametrize("how", [dict(), dict(temperature=0.0), dict(top_k=50), dict(top_p=0.9), dict(min_p=0.05),
                                 dict(top_k=300, top_p=0.8, min_p=0.01, temperature=1.3)], ids=str)
def test_the_mask_is_not_drawn(bd, dtype, vocab, rows, pad, how):
    """The same tokens and log-probabilities, bit for bit, as from logits in which the mask is -inf, wherever it lies."""
    gen = torch.Generator("cuda").manual_seed(vocab + rows)
    # (both with the same strides: sums of log-probabilities go by how a row lies in 16-byte vectors)
    whole = torch.randn((rows, vocab + pad), device="cuda", generator=gen).to(dtype)
    x = whole[:, :vocab]
    u = torch.rand(rows, device="cuda", generator=gen)
    for mask in sorted({0, 1 % vocab, vocab // 3, vocab // 2, vocab - 1}):
        for value in (20.0, math.inf, math.nan, -math.inf, 0.5):
            x[:, mask] = value
            clean = whole.clone()[:, :vocab]
            clean[:, mask] = -math.inf
            want, wlp = bd.bdlm_sample(clean, u, **how)
            token, lp = bd.bdlm_sample(x, u, mask_id=mask, draw_mask=False, **how)
            assert torch.equal(token, want) and torch.equal(lp, wlp), (mask, value)
            now = torch.full((rows,), mask, dtype=torch.int32, device="cuda")
            now[::2] = mask + 1
            out, lp2 = torch.full_like(now, -5), torch.full((rows,), 3.25, device="cuda")
            bd.bdlm_sample(x, u, tokens=now, mask_id=mask, out=out, logprob=lp2, draw_mask=False, **how)
            assert torch.equal(out[1::2], want[1::2]) and torch.equal(lp2[1::2], wlp[1::2]) and torch.all(out[::2] == -5)
    x[:, vocab // 2] = 1.0
    want, wlp = bd.bdlm_sample(x, u, **how)
    for mask in (-1, vocab, -2 ** 31, 2 ** 31 - 1):  # no token of the row
        token, lp = bd.bdlm_sample(x, u, mask_id=mask, draw_mask=False, **how)
        assert torch.equal(token, want) and torch.equal(lp, wlp)


def test_the_exact_sum_leaves_the_mask_out(bd):
    """Equal logits, whose top-p border is met exactly: the sum of all weights is taken anew, without the mask."""
    x = torch.full((6, 301), 2.5, device="cuda").bfloat16()
    x[:, 150] = 9.0
    for p in (0.25, 0.5, 0.75):
        for u in (0.0, 0.5, 1.0):
            token, _ = bd.bdlm_sample(x, torch.full((6,), u, device="cuda"), top_p=p, mask_id=150, draw_mask=False)
            clean = x.double().cpu().numpy()[0].copy()
            clean[150] = -np.inf
            assert token.tolist() == [ao.sample_row(clean, u, top_p=p)[0]] * 6


@pytest.mark.parametrize("how", [dict(temperature=0.0), dict(top_p=0.9), dict()], ids=str)
def test_steps_end_without_masked_rows(bd, how):
    """The mask has the largest logit of every row: a loop until no row is left ends, with the best of the other tokens."""
    from block_diffusion_lm_bdlm_gb300.decode import BlockDecoder

    cache = bd.PageCache.empty(1, 12, 16, 1, 64, 2, 4)
    dec = BlockDecoder(cache, 16)
    dec.begin(dev([16, 16]), check=True)
    gen = torch.Generator("cuda").manual_seed(6)
    mask, vocab = 500, 501
    tokens = torch.full((32,), mask, dtype=torch.int32, device="cuda")
    for step in range(8):
        logits, u = torch.randn(32, vocab, device="cuda", generator=gen), torch.rand(32, device="cuda", generator=gen)
        logits[:, mask] = 30.0
        left = dec.choose(tokens, logits, u, mask, n_min=2, check=True, **how)
        assert left.tolist() == [14 - 2 * step] * 2 == [int((t == mask).sum()) for t in tokens.split(16)]
