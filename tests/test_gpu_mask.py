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
