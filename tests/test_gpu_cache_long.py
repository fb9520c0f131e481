"""The paged 8-bit cache on the GPU where work is split: many sequences and long ones, shares that begin and end
anywhere, units of one and of two MMA tiles side by side, writes whose CTAs take several heads each, and calls at
once. Bounds as in cache_util."""
import numpy as np
import pytest
import torch

from oracle import cache_oracle as co

import cache_util as cu
from test_gpu_cache import attn_case, bd, dev, rows_of  # noqa: F401  (bd is a fixture)

pytestmark = pytest.mark.gpu


def check(bd, c, off, q, qh, block, what="", out=None):
    ref = co.attention(c, 0, qh, off, block, q.shape[2] ** -0.5)
    o, lse = bd.bdlm_cache_attn_fwd(cu.to_device(bd, c), q, dev(off, torch.int32), block, out=out, check=True)
    cu.check_attention(o, lse, ref, what)


# --------------------------------------------------------------- shares and units
def test_every_row_of_many_long_sequences(bd):
    # each CTA's share is many tiles of units with all 256 rows alive
    c, off, q, qh = attn_case(101, [1400 + 37 * s for s in range(24)], [32] * 24, 64, 8, 1, 128, 32)
    check(bd, c, off, q, qh, 32)


@pytest.mark.parametrize("d,page", [(64, 32), (128, 16), (128, 128)])
def test_units_of_one_and_two_tiles_in_a_share(bd, d, page):
    # 4, 128, 240, 256, 260 and 600 flat rows by turns, short and long keys: a share holds several units of both kinds
    rows = [1, 32, 60, 64, 65, 150] * 9
    rng = np.random.default_rng(103)
    lens = [int(r + x) for r, x in zip(rows, rng.integers(0, 700, len(rows)))]
    c, off, q, qh = attn_case(107, lens, rows, page, 4, 1, d, 16)
    check(bd, c, off, q, qh, 16)


def test_more_sequences_than_threads(bd):
    # 1300 sequences (the scan takes 512 at a time), a third of them without rows, some without keys
    rng = np.random.default_rng(109)
    lens = [int(x) for x in rng.integers(0, 90, 1300)]
    rows = [int(min(n, x)) for n, x in zip(lens, rng.choice([0, 1, 4], 1300))]
    c, off, q, qh = attn_case(113, lens, rows, 16, 2, 1, 64, 4)
    check(bd, c, off, q, qh, 4)


@pytest.mark.parametrize("seed", range(10))
def test_random_shapes(bd, seed):
    rng = np.random.default_rng(1000 + seed)
    d, page = int(rng.choice([64, 128])), int(rng.choice([16, 32, 64, 128]))
    Hk, G, block, seqs = int(rng.integers(1, 4)), int(rng.integers(1, 12)), int(rng.integers(1, 70)), int(rng.integers(1, 30))
    lens = [int(np.exp(rng.uniform(0, np.log(1500)))) for _ in range(seqs)]
    rows = [int(rng.integers(0, min(n, 90) + 1)) for n in lens]
    rows[0] = max(rows[0], 1)
    c, off, q, qh = attn_case(2000 + seed, lens, rows, page, G * Hk, Hk, d, block)
    check(bd, c, off, q, qh, block, f"{lens} {rows} page {page} H {G * Hk} Hk {Hk} d {d} block {block}",
          out=None if seed % 2 else torch.empty(q.shape, dtype=torch.float32, device="cuda"))


@pytest.mark.parametrize("rows,dtype", [(1, torch.bfloat16), (9, torch.float32), (40, torch.bfloat16), (64, torch.float32)])
def test_one_long_sequence_of_many_partials(bd, rows, dtype):
    c, off, q, qh = attn_case(127, [30011], [rows], 64, 4, 1, 128, 32)
    check(bd, c, off, q, qh, 32, out=torch.empty(q.shape, dtype=dtype, device="cuda"))


@pytest.mark.parametrize("rows,G", [(5, 3), (100, 3)])
def test_nan_in_a_cut_sequence(bd, rows, G):
    # a NaN value that the last rows alone see, and one that all see, in partials that are merged
    for where in (19990, 700):
        c, off, q, qh = attn_case(131, [20000, 50], [rows, 3], 32, G, 1, 128, 1)
        c["v"][0, c["table"][0, where // 32], 0, where % 32, 77] = 0x7f
        check(bd, c, off, q, qh, 1, f"position {where}")


def test_two_tile_units_whose_scores_grow_and_values_shrink(bd):
    # the running maximum moves in tile after tile, in either half of a tile; then pages of tiny values
    c, off, q, qh = attn_case(137, [1100, 700], [90, 64], 16, 4, 1, 128, 8)
    for s in range(2):
        for j, p in enumerate(c["table"][s][:co.pages_of(c["lens"][s], 16)]):
            c["ks"][0, p] *= 1 + (j if j < 50 else 0)
            c["vs"][0, p] *= 2.0 ** (-70 if j % 7 == 3 else 0)
    check(bd, c, off, q, qh, 8)


def test_a_query_that_is_not_finite_in_a_two_tile_unit(bd):
    c, off, q, qh = attn_case(139, [600], [50], 64, 4, 1, 128, 1)
    ref = co.attention(c, 0, qh, off, 1, 128 ** -0.5)
    for row, head in ((2, 1), (40, 3)):
        q[row, head, 9] = float("inf")
        ref[0][row, head], ref[1][head, row] = np.nan, np.nan
    o, lse = bd.bdlm_cache_attn_fwd(cu.to_device(bd, c), q, dev(off, torch.int32), 1)
    cu.check_attention(o, lse, ref)


@pytest.mark.parametrize("rows", [3, 90])
def test_scores_too_small_for_fp32_hide_masked_keys_all_the_same(bd, rows):
    # queries and key scales whose product underflows: every visible key weighs the same, and no masked key counts
    c, off, q, qh = attn_case(191, [200], [rows], 16, 2, 1, 64, 1)
    q *= 2.0 ** -120
    c["ks"][:] = 2.0 ** -40
    check(bd, c, off, q, q.double().cpu().numpy(), 1)


# --------------------------------------------------------------------- writing
@pytest.mark.parametrize("Hk,page,d,n", [(8, 64, 128, 11000), (3, 128, 64, 30000), (4, 16, 64, 45000)])
def test_write_with_several_heads_per_cta(bd, Hk, page, d, n):
    # enough pages that a CTA takes two or more of a page's heads; the first pages keep rows, some rows are not finite
    rows = [n // 2, 0, n // 3, 7]
    lens = [n // 2 + 5, 9, n // 3, 3 * page + 6]
    c = cu.make(149, lens=[lens[0] % page, 9, 0, lens[3]], page=page, Hk=Hk, d=d, spare=2 + n // page,
                max_pages=co.pages_of(max(lens), page))
    need = [co.pages_of(x, page) for x in lens]
    assert sum(need) <= c["k"].shape[1]
    ids = np.random.default_rng(151).permutation(c["k"].shape[1])
    at = 0
    for s, m in enumerate(need):
        c["table"][s, :m] = ids[at:at + m]
        at += m
    c["lens"][:] = lens
    for x in "kv":  # the kept rows' codes are random: no NaN, so that scales stay as the definition has them
        c[x] &= 0xf7
    rng = np.random.default_rng(157)
    off = cu.offsets(rows)
    k, kh = rows_of(rng, int(off[-1]), Hk, d, 2.0)
    v, vh = rows_of(rng, int(off[-1]), Hk, d, 0.3)
    for row, head, col, x in ((3, 0, 5, np.nan), (n // 4, Hk - 1, d - 1, np.inf), (n // 2 + 70, 1, 0, -np.inf)):
        k[row, head, col], kh[row, head, col] = x, x
        v[row + 1, head, col], vh[row + 1, head, col] = x, x
    cache = cu.to_device(bd, c)
    bd.bdlm_cache_write(cache, k, v, dev(off, torch.int32), check=True)
    co.write(c, 0, kh, vh, off)
    cu.check_same(cu.to_host(cache), c)


def test_write_for_more_sequences_than_one_search_step_splits(bd):
    rng = np.random.default_rng(163)
    lens = [int(x) for x in rng.integers(0, 60, 1500)]
    rows = [int(min(n, x)) for n, x in zip(lens, rng.choice([0, 0, 1, 20], 1500))]
    c = cu.make(167, lens=lens, page=16, Hk=1, d=64)
    off = cu.offsets(rows)
    k, kh = rows_of(rng, int(off[-1]), 1, 64)
    v, vh = rows_of(rng, int(off[-1]), 1, 64)
    cache = cu.to_device(bd, c)
    bd.bdlm_cache_write(cache, k, v, dev(off, torch.int32), check=True)
    co.write(c, 0, kh, vh, off)
    cu.check_same(cu.to_host(cache), c)


# --------------------------------------------------------------- calls at once
def test_calls_at_once_on_two_streams(bd):
    # attention over one layer while another layer is written and read, each stream with workspaces of its own
    c, off, q, qh = attn_case(173, [900, 333, 64], [32, 32, 32], 32, 8, 2, 128, 32, layers=2)
    cache = cu.to_device(bd, c)
    rng = np.random.default_rng(179)
    k, kh = rows_of(rng, 96, 2, 128)
    v, vh = rows_of(rng, 96, 2, 128)
    cu_rows = dev(off, torch.int32)
    torch.cuda.synchronize()
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(4):
        a = bd.bdlm_cache_attn_fwd(cache, q, cu_rows, 32, layer=0, stream=one)
        bd.bdlm_cache_write(cache, k, v, cu_rows, layer=1, stream=two)
        b = bd.bdlm_cache_attn_fwd(cache, q, cu_rows, 32, layer=1, stream=two)
        got.append((a, b))
    torch.cuda.synchronize()
    co.write(c, 1, kh, vh, off)
    cu.check_same(cu.to_host(cache), c)
    refs = [co.attention(c, la, qh, off, 32, 128 ** -0.5) for la in (0, 1)]
    for i, pair in enumerate(got):
        for la in (0, 1):
            cu.check_attention(*pair[la], refs[la], f"turn {i}, layer {la}")


def test_calls_without_a_workspace(bd):
    # small, large, from another current stream, from two threads, small again: the outputs are those of calls with
    # workspaces of their own
    from threading import Thread

    c, off, q, _ = attn_case(211, [3000, 500, 90], [40, 40, 40], 32, 8, 2, 128, 8)
    cache = cu.to_device(bd, c)
    sizes = {}
    for n in (1, 40):
        cu_rows = dev([0, n, 2 * n, 3 * n], torch.int32)
        rows = q[:3 * n].contiguous()
        ws = torch.empty(bd.bdlm_cache_attn_fwd_workspace_bytes(3 * n, 8, 2, 128, 3), dtype=torch.uint8, device="cuda")
        sizes[n] = rows, cu_rows, bd.bdlm_cache_attn_fwd(cache, rows, cu_rows, 8, workspace=ws)
    torch.cuda.synchronize()
    got = []

    def run(n):
        rows, cu_rows, want = sizes[n]
        got.append((bd.bdlm_cache_attn_fwd(cache, rows, cu_rows, 8), want))

    side = torch.cuda.Stream()
    for _ in range(3):
        run(1), run(40)
        with torch.cuda.stream(side):
            run(40), run(1)
    threads = [Thread(target=lambda n=n: [run(n) for _ in range(20)]) for n in (1, 40, 40)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert len(got) == 72
    for (o, lse), want in got:
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


def test_two_graphs_replayed_at_once(bd):
    c, off, q, qh = attn_case(181, [700, 2000], [8, 8], 64, 8, 2, 64, 8)
    cache = cu.to_device(bd, c)
    cu_rows = dev(off, torch.int32)
    ref = co.attention(c, 0, qh, off, 8, 64 ** -0.5)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        bd.bdlm_cache_attn_fwd(cache, q, cu_rows, 8)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(bd.bdlm_cache_attn_fwd(cache, q, cu_rows, 8))
        graphs.append(g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(3):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for o, lse in outs:
        cu.check_attention(o, lse, ref)


def test_a_block_without_room_writes_nothing(bd):
    from block_diffusion_lm_bdlm_gb300.decode import BlockDecoder

    c = cu.make(193, lens=[30, 17], page=16, Hk=1, d=64, spare=1, max_pages=4)
    cache = cu.to_device(bd, c)
    dec = BlockDecoder(cache, 16)
    q = torch.ones(32, 2, 64, dtype=torch.bfloat16, device="cuda")
    out, lse = torch.full_like(q, 5.0), torch.full((2, 32), 5.0, device="cuda")
    assert dec.begin(dev([16, 16], torch.int32)).tolist() == [0, 0, 0]  # two pages would be needed
    dec.attend(0, q, q[:, :1].contiguous(), q[:, :1].contiguous(), out=out, lse=lse)
    assert bool((out == 5).all()) and bool((lse == 5).all())
    cu.check_same(cu.to_host(cache), c)
    with pytest.raises(bd.BDLMError, match="NO_PAGES"):
        dec.begin(dev([16, 16], torch.int32), check=True)
    assert dec.begin(dev([16, 0], torch.int32), check=True).tolist() == [0, 16, 16]


# ---------------------------------------------------------------- large caches
def test_page_calls_on_long_sequences(bd):
    # thousands of pages per sequence: entries are shared out over warps; then shrunk, forked, compacted, written
    c = cu.make(223, lens=[40, 3, 0], page=16, Hk=1, d=64, spare=9000, max_pages=5000, extra_seqs=2)
    cache = cu.to_device(bd, c)
    for lens in ([70000, 33, 0, 0, 0], [70001, 30000, 77, 0, 0], [50000, 30000, 5, 0, 0]):
        bd.bdlm_cache_reserve(cache, dev(lens, torch.int32), check=True)
        assert co.reserve(c, np.array(lens)) == ""
        cu.check_same(cu.to_host(cache), c, str(lens))
    bd.bdlm_cache_fork(cache, dev([0, 1], torch.int32), dev([3, 4], torch.int32), dev([49999, 30000], torch.int32), check=True)
    assert co.fork(c, [0, 1], [3, 4], [49999, 30000]) == ""
    cu.check_same(cu.to_host(cache), c, "fork")
    cache.lens[0], c["lens"][0] = 0, 0
    assert int(bd.bdlm_cache_compact(cache, check=True)) == co.compact(c)
    cu.check_same(cu.to_host(cache), c, "compact")
    bad = cu.to_device(bd, {**c, "table": c["table"].copy()})
    ws = torch.empty(bd.bdlm_cache_pages_workspace_bytes(c["k"].shape[1], 5), dtype=torch.uint8, device="cuda")
    k = torch.ones(40000, 1, 64, dtype=torch.bfloat16, device="cuda")
    rows = dev([0, 0, 20, 20, 40000, 40000], torch.int32)
    bd.bdlm_cache_write(bad, k, k, rows, workspace=ws)
    assert bd.bdlm_read_error(ws) == 0
    bad.table[3, 1000] = -1  # one page in the middle of the 39980 rows
    bd.bdlm_cache_write(bad, k, k, rows, workspace=ws)
    assert bd.bdlm_read_error(ws) == 6
    bd.bdlm_cache_compact(bad, workspace=ws)
    assert bd.bdlm_read_error(ws) == 6


def test_pages_far_beyond_4_gb(bd):
    # 5 GB of keys and of values in two layers, with the used pages at the far end: byte offsets pass 2^32
    page, Hk, d, H, B = 128, 8, 128, 16, 32
    lens, rows = [700, 130, 64], [64, 32, 7]
    c, off, q, qh = attn_case(197, lens, rows, page, H, Hk, d, B)
    n, far = c["k"].shape[1], 19000
    small = cu.to_device(bd, c)
    big = [torch.empty((2, far + n + 4, Hk, page, d), dtype=torch.float8_e4m3fn, device="cuda") for _ in range(2)]
    scales = [torch.ones((2, far + n + 4, Hk), device="cuda") for _ in range(2)]
    for b, s, src, src_s in zip(big, scales, (small.k, small.v), (small.k_scale, small.v_scale)):
        b[1, far:far + n].view(torch.uint8).copy_(src[0].view(torch.uint8))
        s[1, far:far + n] = src_s[0]
    table = torch.zeros((4, 8), dtype=torch.int32, device="cuda")
    table[:3, :small.table.shape[1]] = small.table + far
    cache = bd.PageCache(*big, *scales, table, torch.cat([small.lens, torch.zeros(1, dtype=torch.int32, device="cuda")]))
    cu_rows = dev(list(off) + [off[-1]], torch.int32)
    rng = np.random.default_rng(199)
    (k, kh), (v, vh) = rows_of(rng, int(off[-1]), Hk, d), rows_of(rng, int(off[-1]), Hk, d)

    def back():
        host = {x: c[x].copy() for x in c}
        for x, b, s in (("k", big[0], scales[0]), ("v", big[1], scales[1])):
            host[x][0] = b[1, far:far + n].view(torch.uint8).cpu().numpy()
            host[x + "s"][0] = s[1, far:far + n].double().cpu().numpy()
        return host

    bd.bdlm_cache_write(cache, k, v, cu_rows, layer=1, check=True)
    co.write(c, 0, kh, vh, off)
    cu.check_same(back(), c)
    ref = co.attention(c, 0, qh, off, B, d ** -0.5)
    cu.check_attention(*bd.bdlm_cache_attn_fwd(cache, q, cu_rows, B, layer=1), ref)
    bd.bdlm_cache_fork(cache, dev([0], torch.int32), dev([3], torch.int32), check=True)  # its last page comes to page 0
    o, lse = bd.bdlm_cache_attn_fwd(cache, q[:64].contiguous(), dev([0, 0, 0, 0, 64], torch.int32), B, layer=1)
    cu.check_attention(o, lse, [x[:64] if i in (0, 2) else x[:, :64] for i, x in enumerate(ref)], "forked")
    live = int(bd.bdlm_cache_compact(cache, check=True))
    assert live == sum(co.pages_of(x, page) for x in lens) + 1 and int(cache.table[:3, 0].max()) < live
    cu.check_attention(*bd.bdlm_cache_attn_fwd(cache, q, cu_rows, B, layer=1), ref, "compacted")
