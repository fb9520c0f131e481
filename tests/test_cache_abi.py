"""Refusals of the paged cache's calls on the host: no launch is made (no GPU needed)."""
import ctypes
import os
import re

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INVALID, UNSUP, WS = 1, 2, 3


@pytest.fixture(scope="module")
def bd():
    from block_diffusion_lm_bdlm_gb300 import build

    build.build()
    import block_diffusion_lm_bdlm_gb300 as m

    m.load_library()
    return m


def view(bd, **kw):
    a = dict(k=256, v=512, k_scale=1024, v_scale=2048, table=4096, lens=8192, n_layers=2, n_pages=10, page=64,
             kv_heads=2, head_dim=128, n_seqs=3, max_pages=4, reserved=0)
    a.update(kw)
    return bd._CCache(*[a[f] for f, _ in bd._CCache._fields_])


BAD_CACHES = [(dict(k=None), INVALID), (dict(v=520), INVALID), (dict(k_scale=1025), INVALID), (dict(table=None), INVALID),
              (dict(lens=8194), INVALID), (dict(n_layers=0), INVALID), (dict(n_pages=0), INVALID), (dict(kv_heads=0), INVALID),
              (dict(kv_heads=257), INVALID), (dict(n_seqs=0), INVALID), (dict(n_seqs=65537), INVALID), (dict(max_pages=0), INVALID),
              (dict(max_pages=1 << 25), INVALID), (dict(n_pages=(1 << 26) + 1), INVALID), (dict(reserved=1), INVALID),
              (dict(page=48), UNSUP), (dict(page=256), UNSUP), (dict(head_dim=96), UNSUP)]


def calls(bd):
    lib = bd.load_library()
    big = 1 << 30
    return {
        "write": lambda c, layer=1, k=256, v=256, T=5, cu=64, ws=256, n=big: lib.bdlm_cache_write(c, layer, k, v, T, cu, ws, n, None),
        "attn": lambda c, layer=1, q=256, o=256, lse=64, T=5, H=4, B=16, cu=64, pos=None, dt=0, ws=256, n=big:
            lib.bdlm_cache_attn_fwd(c, layer, q, o, lse, T, H, B, cu, pos, 0.0, dt, ws, n, None),
        "reserve": lambda c, new=64, ws=256, n=big: lib.bdlm_cache_reserve(c, new, ws, n, None),
        "fork": lambda c, p=64, k=64, lens=None, n_forks=2, ws=256, n=big: lib.bdlm_cache_fork(c, p, k, lens, n_forks, ws, n, None),
        "compact": lambda c, live=None, ws=256, n=big: lib.bdlm_cache_compact(c, live, ws, n, None),
    }


@pytest.mark.parametrize("name", ["write", "attn", "reserve", "fork", "compact"])
def test_every_call_checks_the_cache_and_the_workspace(bd, name):
    f = calls(bd)[name]
    for kw, want in BAD_CACHES:
        assert f(view(bd, **kw)) == want, kw
    assert f(None) == INVALID
    assert f(view(bd), ws=None) == WS and f(view(bd), ws=272) == WS and f(view(bd), n=255) == WS
    assert bd.bdlm_last_launch_count() == 0


@pytest.mark.parametrize("name,kw", [
    ("write", dict(layer=2)), ("write", dict(layer=-1)), ("write", dict(k=None)), ("write", dict(v=264)), ("write", dict(T=0)),
    ("write", dict(T=(1 << 30) + 1)), ("write", dict(cu=None)), ("write", dict(cu=66)),
    ("attn", dict(layer=2)), ("attn", dict(q=None)), ("attn", dict(q=264)), ("attn", dict(o=None)), ("attn", dict(lse=66)),
    ("attn", dict(T=0)), ("attn", dict(H=3)), ("attn", dict(H=0)), ("attn", dict(B=0)), ("attn", dict(B=-4)), ("attn", dict(cu=None)),
    ("attn", dict(pos=66)), ("attn", dict(dt=2)), ("attn", dict(T=1 << 30, H=4)),
    ("reserve", dict(new=None)), ("reserve", dict(new=66)),
    ("fork", dict(p=None)), ("fork", dict(k=66)), ("fork", dict(lens=66)), ("fork", dict(n_forks=0)), ("fork", dict(n_forks=4)),
    ("compact", dict(live=66))])
def test_bad_arguments(bd, name, kw):
    assert calls(bd)[name](view(bd), **kw) == INVALID
    assert bd.bdlm_last_launch_count() == 0


def test_workspace_sizes(bd):
    assert bd.bdlm_cache_write_workspace_bytes() == 256
    w = bd.bdlm_cache_attn_fwd_workspace_bytes
    assert w(7, 32, 8, 128, 3) >= 256
    for bad in ((0, 32, 8, 128, 3), (7, 32, 5, 128, 3), (7, 32, 8, 96, 3), (7, 32, 8, 128, 0), (7, 0, 8, 128, 1), (7, 8, 0, 64, 1)):
        assert w(*bad) == 0, bad
    p = bd.bdlm_cache_pages_workspace_bytes
    assert p(100, 4) > p(10, 4) > 256 and p(10, 400) > p(10, 4)
    assert p(0, 4) == 0 and p(10, 0) == 0


def test_status_of_an_exhausted_cache(bd):
    assert bd.status_string(7) == "BDLM_ERR_NO_PAGES"


def test_binding_refuses_host_tensors_and_wrong_shapes(bd):
    f8 = torch.zeros(1, 2, 1, 16, 64, dtype=torch.uint8).view(torch.float8_e4m3fn)
    s = torch.ones(1, 2, 1)
    with pytest.raises(ValueError, match="CUDA"):
        bd.PageCache(f8, f8, s, s, torch.zeros(1, 2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32))


def test_ctypes_struct_matches_the_header(bd, tmp_path):
    import shutil
    import subprocess

    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    names = [f for f, _ in bd._CCache._fields_]
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "bdlm.h"\nint main(void) {\nprintf("%zu\\n", sizeof(bdlm_cache));\n'
                   + "".join(f'printf("%zu\\n", offsetof(bdlm_cache, {f}));\n' for f in names) + "return 0;\n}\n")
    exe = tmp_path / "layout"
    subprocess.run([cc, "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()]
    assert got == [ctypes.sizeof(bd._CCache)] + [getattr(bd._CCache, f).offset for f in names]
    hdr = open(os.path.join(ROOT, "include", "bdlm.h")).read()
    body = hdr[:hdr.index("} bdlm_cache;")]
    body = re.sub(r"/\*.*?\*/", "", body[body.rindex("typedef struct {"):], flags=re.S)
    declared = [x.strip(" *") for line in re.findall(r"(?:void\*|float\*|int32_t\*|int32_t)\s+([\w\s,]+);", body) for x in line.split(",")]
    assert declared == names
