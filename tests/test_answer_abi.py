"""Refusals of the calls that share prefixes, sample and unmask, on the host: no launch is made (no GPU needed)."""
import ctypes

import pytest

from test_cache_abi import BAD_CACHES, INVALID, UNSUP, WS, bd, view  # noqa: F401  (bd is a fixture)

BIG = 1 << 30


def shared(bd, c, layer=1, q=256, o=256, lse=64, T=5, H=4, B=16, cu=64, pos=None, runs=64, dt=0, ws=256, n=BIG):
    return bd.load_library().bdlm_cache_attn_shared_fwd(c, layer, q, o, lse, T, H, B, cu, pos, runs, 0.0, dt, ws, n, None)


def prefixes(bd, c, T=5, cu=64, pos=None, runs=128, ws=256, n=BIG):
    return bd.load_library().bdlm_cache_prefixes(c, T, cu, pos, runs, ws, n, None)


@pytest.mark.parametrize("call", [shared, prefixes])
def test_caches_and_workspaces(bd, call):
    for kw, want in BAD_CACHES:
        assert call(bd, view(bd, **kw)) == want, kw
    assert call(bd, None) == INVALID
    assert call(bd, view(bd), ws=None) == WS and call(bd, view(bd), ws=272) == WS and call(bd, view(bd), n=255) == WS
    assert bd.bdlm_last_launch_count() == 0


@pytest.mark.parametrize("kw", [dict(runs=None), dict(runs=66), dict(q=None), dict(o=264), dict(lse=None), dict(cu=None), dict(pos=2),
                                dict(T=0), dict(T=-1), dict(H=3), dict(H=0), dict(B=0), dict(dt=2), dict(layer=2), dict(layer=-1)])
def test_shared_attention(bd, kw):
    assert shared(bd, view(bd), **kw) == INVALID


# view(bd): 3 sequences of 4 entries: table is [4096, 4144), lens [8192, 8204); runs takes 36 bytes, cu_rows 16, q_pos 12
@pytest.mark.parametrize("kw", [dict(cu=None), dict(cu=65), dict(pos=2), dict(runs=None), dict(runs=129), dict(T=-1), dict(T=(1 << 30) + 1),
                                dict(runs=4064), dict(runs=4140), dict(runs=8160), dict(runs=8200), dict(runs=76), dict(runs=32),
                                dict(pos=160), dict(pos=120)])
def test_prefixes(bd, kw):
    assert prefixes(bd, view(bd), **kw) == INVALID


def test_prefixes_sizes(bd):
    assert prefixes(bd, view(bd, n_seqs=16385, max_pages=1, lens=1 << 20), runs=1 << 24) == UNSUP
    assert bd.bdlm_cache_prefixes_workspace_bytes(16384) > 0 == bd.bdlm_cache_prefixes_workspace_bytes(16385)
    assert bd.bdlm_cache_prefixes_workspace_bytes(0) == 0
    f = bd.bdlm_cache_attn_shared_fwd_workspace_bytes
    assert f(5, 4, 2, 64, 3) > bd.bdlm_cache_attn_fwd_workspace_bytes(5, 4, 2, 64, 3) > 0
    assert f(0, 4, 2, 64, 3) == f(5, 4, 3, 64, 3) == f(5, 4, 2, 96, 3) == f(5, 4, 2, 64, 0) == 0


def sample(bd, x=1 << 20, dt=0, rows=4, V=100, stride=100, u=64, how=(None, None, None, None), tokens=None, token=128, lp=256):
    h = None if how is None else ctypes.byref(bd._CSampling(*how, 1.0, 0, 1.0, 0.0))
    return bd.load_library().bdlm_sample(x, dt, rows, V, stride, u, h, tokens, 7, token, lp, None)


@pytest.mark.parametrize("kw", [dict(x=None), dict(x=257), dict(x=258, dt=1), dict(dt=3), dict(dt=-1), dict(rows=0), dict(rows=-1),
                                dict(rows=(1 << 26) + 1), dict(V=0), dict(V=-5), dict(stride=99), dict(stride=-100), dict(stride=1 << 41),
                                dict(u=None), dict(u=66), dict(how=None), dict(how=(2, None, None, None)), dict(how=(None, 3, None, None)),
                                dict(how=(None, None, 5, None)), dict(how=(None, None, None, 1)), dict(tokens=6), dict(token=None),
                                dict(token=130), dict(lp=None), dict(lp=259), dict(token=64), dict(token=72), dict(lp=140), dict(lp=52),
                                dict(how=(120, None, None, None)), dict(how=(None, 260, None, None)), dict(tokens=132), dict(tokens=256),
                                dict(x=100), dict(lp=(1 << 20) + 700)])
def test_sample(bd, kw):
    assert sample(bd, **kw) == INVALID and bd.bdlm_last_launch_count() == 0


def test_sample_vocabulary(bd):
    assert sample(bd, V=(1 << 18) + 1, stride=1 << 20, x=1 << 30) == UNSUP


def unmask(bd, tokens=256, sampled=512, lp=1024, T=5, cu=2048, n=2, k=None, thr=None, out=4096, left=8192, ws=256, bytes=256):
    return bd.load_library().bdlm_unmask(tokens, sampled, lp, T, cu, n, 7, k, 0, thr, 0.0, out, left, ws, bytes, None)


@pytest.mark.parametrize("kw", [dict(tokens=None), dict(sampled=513), dict(lp=None), dict(cu=None), dict(cu=2050), dict(k=2), dict(thr=1),
                                dict(out=None), dict(left=None), dict(left=8193), dict(T=0), dict(T=(1 << 30) + 1), dict(n=0), dict(n=65537),
                                dict(out=260), dict(out=512), dict(out=1036), dict(out=2044), dict(left=4100), dict(left=272), dict(left=520),
                                dict(left=1040), dict(left=2056), dict(k=4100), dict(thr=8196), dict(k=8188)])
def test_unmask(bd, kw):
    assert unmask(bd, **kw) == INVALID and bd.bdlm_last_launch_count() == 0


def test_unmask_workspace(bd):
    assert bd.bdlm_unmask_workspace_bytes() == 256
    assert unmask(bd, ws=264) == WS and unmask(bd, bytes=255) == WS
    assert unmask(bd, out=256, bytes=255) == WS  # in place passes on to the next check


def test_bindings_refuse_host_tensors(bd):
    import torch

    with pytest.raises(ValueError):
        bd.bdlm_sample(torch.zeros(2, 5), torch.zeros(2))
    with pytest.raises(ValueError):
        bd.bdlm_unmask(torch.zeros(2, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), torch.zeros(2),
                       torch.zeros(2, dtype=torch.int32), 7)


def test_sampling_flags(bd):
    """Flags that there are not, and a reserved word that is set, are refused."""
    for more in ((2, 0), (-1, 0), (1 << 31 - 1, 0), (0, 1), (1, -1)):
        h = ctypes.byref(bd._CSampling(None, None, None, None, 1.0, 0, 1.0, 0.0, *more))
        assert bd.load_library().bdlm_sample(1 << 20, 0, 4, 100, 100, 64, h, None, 7, 128, 256, None) == INVALID
    assert ctypes.sizeof(bd._CSampling) == 56
