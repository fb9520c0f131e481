"""Log-probabilities of tokens far below the largest logit: 2^-17 and one rounding to fp32 (test_gpu_sample)."""
import numpy as np
import pytest
import torch

from test_gpu_sample import DTYPES, bd, check  # noqa: F401  (bd is a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("least", [130.0, 1026.0, 16400.0])
def test_far_tokens_round_once(bd, dtype, least):
    """Just above a power of two a rounding is off by up to 2^-24 of the value, and the distance to the largest logit is one value
    that would be rounded before the sum's logarithm comes off."""
    rng = np.random.default_rng(int(least))
    x = -least * rng.uniform(1.0, 1.06, (400, 50))
    x[:, 17:22] = rng.uniform(-3, 3, (400, 5))
    check(bd, torch.from_numpy(x).to(DTYPES[dtype]).cuda(), torch.rand(400, generator=torch.Generator("cuda").manual_seed(1), device="cuda"),
          temperature=1e7)
