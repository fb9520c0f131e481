"""Attention over the paged cache cut into another number of shares than one per SM: from one, which leaves the merge
nothing to do, to as many as the workspace has room for. And caches over which a tile that is lost or counted twice at a
cut would show (cache_marks)."""
import ctypes
import os
import subprocess

import numpy as np
import pytest
import torch

from oracle import cache_oracle as co

import cache_marks as cm
import cache_util as cu
from test_gpu_cache import attn_case, bd, dev  # noqa: F401  (bd is a fixture)

pytestmark = pytest.mark.gpu
HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def with_ctas(bd, tmp_path_factory):
    """attention(cache, q, cu_rows, block, ctas, f32) -> (o, lse), in a workspace filled with 0xff"""
    from block_diffusion_lm_bdlm_gb300 import build as b

    so = str(tmp_path_factory.mktemp("ctas") / "attn_ctas.so")
    objs = [os.path.join(b.BUILD, f) for f in ("cache_attn.o", "cache_attn_d64.o", "cache_attn_d128.o")]
    subprocess.run([b.nvcc(), *b.ARCH, *b.NVCC_FLAGS, "-shared", os.path.join(HERE, "attn_ctas.cu"), *objs, "-o", so], check=True)
    f = ctypes.CDLL(so).attn_with_ctas
    vp, i32 = ctypes.c_void_p, ctypes.c_int32
    f.argtypes = [vp, vp, vp, vp, ctypes.c_longlong, i32, i32, vp, i32, vp, i32, vp]

    def attention(cache, q, cu_rows, block, ctas, f32=False):
        assert 1 <= ctas <= 256
        T, H, d = q.shape
        ws = torch.full((bd.bdlm_cache_attn_fwd_workspace_bytes(T, H, cache.kv_heads, d, cache.n_seqs),), 255,
                        dtype=torch.uint8, device="cuda")
        o = torch.empty(q.shape, dtype=torch.float32 if f32 else torch.bfloat16, device="cuda")
        lse = torch.empty((H, T), dtype=torch.float32, device="cuda")
        st = f(ctypes.addressof(cache.c), q.data_ptr(), o.data_ptr(), lse.data_ptr(), T, H, block, cu_rows.data_ptr(), int(f32),
               ws.data_ptr(), ctas, torch.cuda.current_stream().cuda_stream)
        assert st == 0 and bd.bdlm_read_error(ws) == 0
        return o, lse

    return attention


@pytest.mark.parametrize("d,page,G,rows", [(64, 16, 4, [3, 1, 20, 0, 50]), (128, 64, 4, [40, 70, 1, 0, 33])])
def test_any_number_of_shares_gives_the_same_attention(with_ctas, bd, d, page, G, rows):
    c, off, q, qh = attn_case(503, [500, 129, 1000, 0, 257], rows, page, 2 * G, 2, d, 16)
    ref = co.attention(c, 0, qh, off, 16, d ** -0.5)
    cache = cu.to_device(bd, c)
    for ctas in (1, 2, 3, 7, 16, 61, 151, 256):
        o, lse = with_ctas(cache, q, dev(off, torch.int32), 16, ctas, f32=ctas % 2 == 0)
        cu.check_attention(o, lse, ref, f"{ctas} shares")


@pytest.mark.parametrize("keys", ["any", "alike"])
@pytest.mark.parametrize("name", list(cm.CASES))
def test_no_tile_is_lost_or_counted_twice(with_ctas, bd, name, keys):
    block, d = cm.CASES[name][6], cm.CASES[name][5]
    c, off, q, qh = cm.make(name, keys)
    ref = co.attention(c, 0, qh, off, block, d ** -0.5)
    cache, q, cu_rows = cu.to_device(bd, c), q.cuda(), dev(off, torch.int32)
    cu.check_attention(*bd.bdlm_cache_attn_fwd(cache, q, cu_rows, block, check=True), ref)
    out = torch.empty(q.shape, dtype=torch.float32, device="cuda")
    cu.check_attention(*bd.bdlm_cache_attn_fwd(cache, q, cu_rows, block, out=out), ref)
    for ctas in (1, 7, 61, 200, 256):
        cu.check_attention(*with_ctas(cache, q, cu_rows, block, ctas, f32=ctas % 2 == 0), ref, f"{ctas} shares")
