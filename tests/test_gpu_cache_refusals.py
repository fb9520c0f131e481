"""Page calls that refuse an item in their last check, where every CTA of the plan's cluster has items of its own: they
leave the cache as it was, and the next call works."""
import numpy as np
import pytest
import torch

from oracle import cache_oracle as co

import cache_util as cu
from test_gpu_cache import attn_case, bd, dev  # noqa: F401  (bd is a fixture)

pytestmark = pytest.mark.gpu


def shared_pairs(n):
    """n parents of 20 positions and n children that share page 0 of theirs and stop inside it: none may grow."""
    c = cu.make(301, lens=[20] * n, page=16, Hk=1, d=64, spare=4 * n, max_pages=4, extra_seqs=n)
    assert co.fork(c, list(range(n)), list(range(n, 2 * n))) == ""
    c["lens"][n:] = 9
    return c


@pytest.mark.parametrize("who", ["one", "every eighth", "all"])
def test_growth_inside_shared_pages_is_refused_wherever_it_is_asked_for(bd, who):
    n = 1200
    c = shared_pairs(n)
    cache = cu.to_device(bd, c)
    ws = torch.empty(bd.bdlm_cache_pages_workspace_bytes(c["k"].shape[1], 2 * n), dtype=torch.uint8, device="cuda")
    grow = {"one": [2 * n - 1], "every eighth": range(n, 2 * n, n // 8), "all": range(n, 2 * n)}[who]
    want = c["lens"].copy()
    want[list(grow)] += 1
    new = dev(want, torch.int32)
    for _ in range(50):
        bd.bdlm_cache_reserve(cache, new, workspace=ws)
    assert bd.bdlm_read_error(ws) == 6
    cu.check_same(cu.to_host(cache), c)
    info = int(ws[4:8].view(torch.int32))
    assert info in grow
    want[n:] = 0
    bd.bdlm_cache_reserve(cache, dev(want, torch.int32), workspace=ws)
    assert bd.bdlm_read_error(ws) == 0 and co.reserve(c, want) == ""
    cu.check_same(cu.to_host(cache), c)


@pytest.mark.parametrize("n", [1, 8, 3000])
def test_a_parent_that_is_a_child_of_the_same_call_is_refused(bd, n):
    c = cu.make(307, lens=[20], page=16, Hk=1, d=64, spare=2 * n + 4, max_pages=4, extra_seqs=2 * n)
    cache = cu.to_device(bd, c)
    ws = torch.empty(bd.bdlm_cache_pages_workspace_bytes(c["k"].shape[1], 2 * n + 1), dtype=torch.uint8, device="cuda")
    # every second fork takes the child of the one before as its parent
    parents = dev([x for i in range(n) for x in (0, 1 + 2 * i)], torch.int32)
    children = dev(list(range(1, 2 * n + 1)), torch.int32)
    for _ in range(50):
        bd.bdlm_cache_fork(cache, parents, children, workspace=ws)
    assert bd.bdlm_read_error(ws) == 6
    cu.check_same(cu.to_host(cache), c)
    parents.zero_()
    bd.bdlm_cache_fork(cache, parents, children, workspace=ws)
    assert bd.bdlm_read_error(ws) == 0 and co.fork(c, [0] * 2 * n, list(range(1, 2 * n + 1))) == ""
    cu.check_same(cu.to_host(cache), c)


def test_a_block_size_beyond_32_bits_is_refused(bd):
    c, off, q, qh = attn_case(311, [90], [6], 16, 4, 2, 64, 1)
    cache = cu.to_device(bd, c)
    for block in (2 ** 32 + 1, 2 ** 31, -2 ** 32 + 4):  # modulo 2^32 two of them would be taken as 1 and 4
        with pytest.raises(bd.BDLMError):
            bd.bdlm_cache_attn_fwd(cache, q, dev(off, torch.int32), block)
    o, lse = bd.bdlm_cache_attn_fwd(cache, q, dev(off, torch.int32), 2 ** 31 - 1)  # every key is seen
    cu.check_attention(o, lse, co.attention(c, 0, qh, off, 2 ** 31 - 1, 0.125))


def test_fork_lengths_that_lie_in_the_lengths(bd):
    # those of the parents themselves are fine; one that the same call sets (a child's) is refused
    c = cu.make(313, lens=[20, 33], page=16, Hk=1, d=64, spare=12, max_pages=4, extra_seqs=4)
    cache = cu.to_device(bd, c)
    ws = torch.empty(bd.bdlm_cache_pages_workspace_bytes(c["k"].shape[1], 6), dtype=torch.uint8, device="cuda")
    for _ in range(20):
        bd.bdlm_cache_fork(cache, dev([1, 1], torch.int32), dev([2, 3], torch.int32), cache.lens[1:3], workspace=ws)
    assert bd.bdlm_read_error(ws) == 6
    cu.check_same(cu.to_host(cache), c)
    bd.bdlm_cache_fork(cache, dev([0, 1], torch.int32), dev([2, 3], torch.int32), cache.lens[:2], check=True)
    assert co.fork(c, [0, 1], [2, 3]) == ""
    cu.check_same(cu.to_host(cache), c)
    bd.bdlm_cache_reserve(cache, cache.lens, check=True)
    cu.check_same(cu.to_host(cache), c)
