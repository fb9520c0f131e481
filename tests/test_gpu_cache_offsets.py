"""Weights held under a row's moving offset: what was stored before the offset moved keeps its bits."""
import numpy as np
import pytest
import torch

from oracle import cache_oracle as co

import cache_util as cu
from test_gpu_cache import bd, dev  # noqa: F401  (bd is a fixture)

pytestmark = pytest.mark.gpu


def code(x):
    return int(co.encode(np.array([x]))[0])


@pytest.mark.parametrize("up", [16, 24, 26, 28])
@pytest.mark.parametrize("page,rows,d", [(64, 64, 128), (16, 40, 128), (64, 50, 64), (64, 3, 128)])
def test_the_half_tile_before_an_offset_moves_far(bd, page, rows, d, up):
    # Base-2 scores of about 0 but for key A (10, in the first half of the second tile, which fits the first tile's
    # offset) and key B (`up`, in its second half, which moves the offset by 2^-up): A weighs 2^(10 - up) of B, and
    # column 1 holds A's value alone. With an offset that leaves B at most 2^4, A lies at 2^(14 - up) or more: at least
    # 2^-15, where fp16 is off by 2^-10 of it at most; the bound of cache_util allows more than 4 percent.
    G, block = 4, 256
    c = cu.make(601, lens=[256], page=page, Hk=1, d=d)
    c["k"][:], c["v"][:], c["ks"][:], c["vs"][:] = 0, 0, 1.0, 1.0
    at = lambda key: (0, c["table"][0, key // page], 0, key % page)
    c["k"][at(128 + 20)][0], c["k"][at(128 + 90)][0] = code(10.0), code(float(up))
    c["v"][at(128 + 20)][1], c["v"][at(128 + 90)][0] = code(448.0), code(1.0)
    q = torch.zeros(rows, G, d, dtype=torch.bfloat16)
    q[:, :, 0] = d ** 0.5 * np.log(2.0)
    qh = q.double().numpy()
    ref = co.attention(c, 0, qh, [0, rows], block, d ** -0.5)
    o, lse = bd.bdlm_cache_attn_fwd(cu.to_device(bd, c), q.cuda(), dev([0, rows], torch.int32), block,
                                    out=torch.empty(q.shape, dtype=torch.float32, device="cuda"))
    cu.check_attention(o, lse, ref)


@pytest.mark.parametrize("up", [24, 26])
@pytest.mark.parametrize("page,rows", [(64, 64), (16, 40)])
def test_the_first_half_of_a_first_tile(bd, page, rows, up):
    # the same within the first tile: A (0) lies at 2^4 before B moves the offset, and afterwards at 2^(4 - up) or half of
    # that, which fp16 holds exactly down to 2^-24
    d, G = 128, 4
    c = cu.make(607, lens=[128], page=page, Hk=1, d=d)
    c["k"][:], c["v"][:], c["ks"][:], c["vs"][:] = 0, 0, 1.0, 1.0
    at = lambda key: (0, c["table"][0, key // page], 0, key % page)
    c["k"][at(90)][0], c["v"][at(90)][0], c["v"][at(20)][1] = code(float(up)), code(1.0), code(448.0)
    q = torch.zeros(rows, G, d, dtype=torch.bfloat16)
    q[:, :, 0] = d ** 0.5 * np.log(2.0)
    qh = q.double().numpy()
    ref = co.attention(c, 0, qh, [0, rows], 256, d ** -0.5)
    o, lse = bd.bdlm_cache_attn_fwd(cu.to_device(bd, c), q.cuda(), dev([0, rows], torch.int32), 256,
                                    out=torch.empty(q.shape, dtype=torch.float32, device="cuda"))
    cu.check_attention(o, lse, ref)
