"""The paged 8-bit cache on the GPU against the float64 oracle: writing, attention, the page calls, and
all of them together (cache_util holds the error bounds and what they count)."""
import numpy as np
import pytest
import torch

from oracle import cache_oracle as co

import cache_util as cu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def bd():
    import block_diffusion_lm_bdlm_gb300 as m

    m.load_library()
    return m


def dev(x, dtype):
    return torch.as_tensor(np.asarray(x)).to("cuda", dtype)


def rows_of(rng, T, Hk, d, std=1.0):
    x = torch.from_numpy(rng.standard_normal((T, Hk, d)) * std).bfloat16()
    return x.cuda(), x.double().numpy()


# ------------------------------------------------------------------- writing
WRITES = [
    # lens (with the new rows), rows, page, Hk, d
    ([1], [1], 16, 1, 64),
    ([5, 16, 17, 33], [5, 16, 17, 33], 16, 3, 64),
    ([100, 64, 0, 65, 200], [1, 64, 0, 2, 37], 64, 2, 128),
    ([300, 129, 128, 127], [300, 1, 128, 126], 128, 8, 128),
    ([33, 31, 64, 90], [2, 31, 33, 59], 32, 2, 64),
    ([700, 3, 260], [650, 2, 7], 32, 1, 128),
    ([40] * 70, list(range(40)) + [3] * 30, 16, 1, 128),
]


@pytest.mark.parametrize("lens,rows,page,Hk,d", WRITES)
def test_write(bd, lens, rows, page, Hk, d):
    c = cu.make(len(lens) + page, lens=lens, page=page, Hk=Hk, d=d, layers=2, max_pages=co.pages_of(max(lens), page) + 1)
    rng = np.random.default_rng(1)
    off = cu.offsets(rows)
    T = int(off[-1]) + 3  # rows behind the last sequence
    k, kh = rows_of(rng, T, Hk, d, 3.0)
    v, vh = rows_of(rng, T, Hk, d, 0.01)
    cache = cu.to_device(bd, c)
    bd.bdlm_cache_write(cache, k, v, dev(off, torch.int32), layer=1, check=True)
    co.write(c, 1, kh, vh, off)
    cu.check_same(cu.to_host(cache), c)


@pytest.mark.parametrize("kind", ["zeros", "tiny", "huge", "nan", "inf", "ties"])
def test_write_values(bd, kind):
    c = cu.make(3, lens=[23, 40], page=16, Hk=2, d=64)
    rng = np.random.default_rng(2)
    off = [0, 10, 30]
    x = rng.standard_normal((30, 2, 64))
    if kind == "zeros":
        x[:] = 0
    if kind == "tiny":
        x *= 2.0 ** -130
    if kind == "huge":
        x *= 2.0 ** 125
    if kind == "nan":
        x[3, 1, 5] = np.nan
        x[12] = np.nan
    if kind == "inf":
        x[3, 0, 5], x[20, 1, 7] = np.inf, -np.inf
    if kind == "ties":
        x = rng.integers(-127, 128, x.shape) / 16.0  # 8-bit values: many lie halfway between codes
        x[0, 0, 0] = 448.0
    x = torch.from_numpy(x).bfloat16()
    cache = cu.to_device(bd, c)
    bd.bdlm_cache_write(cache, x.cuda(), (-x).cuda(), dev(off, torch.int32), check=True)
    co.write(c, 0, x.double().numpy(), -x.double().numpy(), off)
    cu.check_same(cu.to_host(cache), c)


def test_write_again_with_smaller_and_larger_rows(bd):
    c = cu.make(4, lens=[50], page=32, Hk=1, d=128, max_pages=4)
    cache = cu.to_device(bd, c)
    rng = np.random.default_rng(3)
    for std in (1.0, 40.0, 0.02):
        k, kh = rows_of(rng, 20, 1, 128, std)
        bd.bdlm_cache_write(cache, k, k, dev([0, 20], torch.int32), check=True)
        co.write(c, 0, kh, kh, [0, 20])
        cu.check_same(cu.to_host(cache), c, f"std {std}")


def test_write_skips_bad_sequences(bd):
    c = cu.make(5, lens=[20, 20, 20, 20], page=16, Hk=1, d=64, max_pages=3)
    rng = np.random.default_rng(4)
    k, kh = rows_of(rng, 16, 1, 64)
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    for what in ("page", "length", "rows"):
        bad = {x: y.copy() for x, y in c.items()}
        off = np.array([0, 4, 8, 12, 16])
        if what == "page":
            bad["table"][1, 1] = 1000
        if what == "length":
            bad["lens"][1] = 49  # more than the table holds
        if what == "rows":
            bad["lens"][1] = 3  # fewer than its new rows
        cache = cu.to_device(bd, bad)
        bd.bdlm_cache_write(cache, k, k, dev(off, torch.int32), workspace=ws)
        assert bd.bdlm_read_error(ws) == 6
        want = {x: y.copy() for x, y in c.items()}
        part = dict(want, lens=np.delete(c["lens"], 1), table=np.delete(c["table"], 1, 0))
        co.write(part, 0, np.delete(kh, slice(4, 8), 0), np.delete(kh, slice(4, 8), 0), [0, 4, 8, 12])
        got = cu.to_host(cache)
        for name in ("k", "v"):
            assert cu.same_codes(got[name], want[name]), what
        assert np.array_equal(got["ks"], want["ks"])


# ----------------------------------------------------------------- attention
ATTN = [
    # lens, rows, page, H, Hk, d, block
    ([1], [1], 16, 1, 1, 64, 1),
    ([600], [1], 16, 16, 4, 64, 1),
    ([127, 128, 129, 1, 0], [1, 1, 1, 1, 0], 64, 8, 2, 128, 1),
    ([515, 32, 96, 1000], [32, 32, 32, 32], 64, 8, 2, 128, 32),
    ([300], [64], 128, 4, 1, 128, 64),
    ([300, 40], [300, 40], 32, 4, 2, 128, 1),
    ([530], [530], 128, 8, 2, 128, 48),
    ([400, 70], [400, 33], 16, 6, 2, 64, 16),
    ([257, 3, 90], [5, 3, 47], 16, 12, 4, 64, 16),
    ([700], [9], 32, 35, 5, 128, 7),
    ([1500, 2100], [3, 1], 128, 32, 2, 64, 4),
    ([200], [200], 64, 3, 3, 64, 1000),
    ([260] * 40, [2] * 40, 16, 2, 1, 128, 3),
]


def attn_case(seed, lens, rows, page, H, Hk, d, block, **kw):
    c = cu.make(seed, lens=lens, page=page, Hk=Hk, d=d, **kw)
    off = cu.offsets(rows)
    q, qh = rows_of(np.random.default_rng(seed + 1), int(off[-1]), H, d, 1.5)
    return c, off, q, qh


@pytest.mark.parametrize("lens,rows,page,H,Hk,d,block", ATTN)
def test_attention(bd, lens, rows, page, H, Hk, d, block):
    c, off, q, qh = attn_case(7 * len(lens) + page, lens, rows, page, H, Hk, d, block)
    ref = co.attention(c, 0, qh, off, block, d ** -0.5)
    cache = cu.to_device(bd, c)
    for dtype in (torch.bfloat16, torch.float32):
        out = torch.full(q.shape, 9.0, dtype=dtype, device="cuda")
        o, lse = bd.bdlm_cache_attn_fwd(cache, q, dev(off, torch.int32), block, out=out, check=True)
        cu.check_attention(o, lse, ref, str(dtype))


@pytest.mark.parametrize("d", [64, 128])
def test_attention_with_positions_gives_partials(bd, d):
    # the keys of one sequence split over two caches (the rows themselves are in neither): the merge of the partials
    # is the attention over all keys; a cache of length 0 gives o = 0, lse = -inf
    page, H, Hk, n, cut, B = 32, 8, 2, 333, 160, 16
    c, off, q, qh = attn_case(11, [n], [20], page, H, Hk, d, B)
    one = {**c, "table": c["table"][:, :cut // page], "lens": np.array([cut])}
    two = {**c, "table": c["table"][:, cut // page:], "lens": np.array([n - cut])}
    parts = []
    for part, pos in ((one, n), (two, n - cut), ({**one, "lens": np.array([0])}, n)):
        ref = co.attention(part, 0, qh, off, B, d ** -0.5, q_pos=[pos])
        out = torch.empty(q.shape, dtype=torch.float32, device="cuda")
        o, lse = bd.bdlm_cache_attn_fwd(cu.to_device(bd, part), q, dev(off, torch.int32), B, q_pos=dev([pos], torch.int32),
                                        out=out, check=True)
        cu.check_attention(o, lse, ref)
        parts.append((o, lse))
    o, lse = bd.bdlm_lse_merge([p[0] for p in parts], [p[1] for p in parts])
    full = co.attention(c, 0, qh, off, B, d ** -0.5, q_pos=[n])
    cu.check_attention(o, lse, (full[0], full[1], full[2], 2 * full[3], 2 * full[4]), "merged")  # two partials' errors


def test_attention_rows_inside_the_first_blocks_see_part_of_the_cache(bd):
    c, off, q, qh = attn_case(13, [50, 20], [6, 3], 16, 4, 2, 64, 8)
    ref = co.attention(c, 0, qh, off, 8, 0.125, q_pos=[5, 40])
    o, lse = bd.bdlm_cache_attn_fwd(cu.to_device(bd, c), q, dev(off, torch.int32), 8, q_pos=dev([5, 40], torch.int32))
    cu.check_attention(o, lse, ref)


def test_attention_softmax_scale(bd):
    c, off, q, qh = attn_case(17, [150], [4], 16, 4, 2, 64, 4)
    ref = co.attention(c, 0, qh, off, 4, 0.3)
    cache = cu.to_device(bd, c)
    cu.check_attention(*bd.bdlm_cache_attn_fwd(cache, q, dev(off, torch.int32), 4, softmax_scale=0.3), ref)
    a = bd.bdlm_cache_attn_fwd(cache, q, dev(off, torch.int32), 4)
    b = bd.bdlm_cache_attn_fwd(cache, q, dev(off, torch.int32), 4, softmax_scale=-1.0)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_attention_leaves_rows_behind_the_last_sequence(bd):
    c, off, q, qh = attn_case(19, [40, 9], [3, 2], 16, 4, 2, 64, 4)
    pad = torch.cat([q, torch.full((5, 4, 64), float("nan"), dtype=torch.bfloat16, device="cuda")])
    out = torch.full(pad.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((4, 10), 7.0, device="cuda")
    bd.bdlm_cache_attn_fwd(cu.to_device(bd, c), pad, dev(off, torch.int32), 4, out=out, lse=lse, check=True)
    assert bool((out[5:] == 7).all()) and bool((lse[:, 5:] == 7).all())
    cu.check_attention(out[:5], lse[:, :5].contiguous(), co.attention(c, 0, qh, off, 4, 0.125))


@pytest.mark.parametrize("d,page,block,G", [(64, 16, 1, 2), (128, 64, 24, 4), (128, 128, 1, 1), (64, 128, 5, 8)])
def test_nan_reaches_only_the_rows_that_see_it(bd, d, page, block, G):
    # NaN codes in keys and values at a position that some rows of a tile see and others do not; the rows of other
    # sequences and the stale rows of pages (random codes, NaN among them) must not feel it either
    n, r = 300, 300
    for where, name in ((150, "v"), (150, "k"), (299, "v"), (128, "v")):
        c, off, q, qh = attn_case(23, [n, 77], [r, 5], page, 2 * G, 2, d, block)
        c[name][0, c["table"][0, where // page], 1, where % page, 3] = 0xff if name == "v" else 0x7f
        ref = co.attention(c, 0, qh, off, block, d ** -0.5)
        o, lse = bd.bdlm_cache_attn_fwd(cu.to_device(bd, c), q, dev(off, torch.int32), block)
        if name == "v":
            assert np.isnan(ref[0]).any() and not np.isnan(ref[0]).all()
        cu.check_attention(o, lse, ref, f"{name} {where}")


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_a_query_that_is_not_finite_spoils_its_row_alone(bd, value):
    c, off, q, qh = attn_case(29, [150], [6], 16, 4, 2, 64, 1)
    q[2, 1, 7] = value
    clean = co.attention(c, 0, qh, off, 1, 0.125)
    o, lse = bd.bdlm_cache_attn_fwd(cu.to_device(bd, c), q, dev(off, torch.int32), 1)
    clean[0][2, 1], clean[1][1, 2] = np.nan, np.nan
    cu.check_attention(o, lse, clean)


@pytest.mark.parametrize("d", [64, 128])
def test_pages_of_very_unlike_magnitude(bd, d):
    # scales 2^40 apart between the pages of one sequence, for keys and for values: tiny values still count where
    # their keys carry the weight
    c, off, q, qh = attn_case(31, [500], [3], 16, 4, 1, d, 1, page_spread=0.0)
    ids = c["table"][0]
    c["vs"][0, ids[:10]] *= 2.0 ** 20
    c["vs"][0, ids[20:]] *= 2.0 ** -20
    c["ks"][0, ids[5:]] *= 2.0 ** -30
    ref = co.attention(c, 0, qh, off, 1, d ** -0.5)
    o, lse = bd.bdlm_cache_attn_fwd(cu.to_device(bd, c), q, dev(off, torch.int32), 1)
    cu.check_attention(o, lse, ref)


def test_scales_that_are_not_powers_of_two(bd):
    c, off, q, qh = attn_case(37, [333, 40], [33, 2], 32, 4, 2, 128, 16)
    rng = np.random.default_rng(5)
    for x in ("ks", "vs"):
        c[x] = (c[x] * rng.uniform(0.5, 1.0, c[x].shape)).astype(np.float32).astype(np.float64)
    ref = co.attention(c, 0, qh, off, 16, 128 ** -0.5)
    cu.check_attention(*bd.bdlm_cache_attn_fwd(cu.to_device(bd, c), q, dev(off, torch.int32), 16), ref)


@pytest.mark.parametrize("n", [4000, 40000])
def test_one_key_holds_half_the_weight(bd, n):
    # one key's score lies ln(n) above all others, which share the other half: their small weights must not be lost
    d, page = 128, 64
    c = cu.make(41, lens=[n], page=page, Hk=1, d=d)
    c["k"][:], c["ks"][:] = 0, 1.0
    c["k"][0, c["table"][0, 0], 0, 3, 0] = 0x38  # 1.0
    q = torch.zeros(2, 2, d, dtype=torch.bfloat16, device="cuda")
    q[:, :, 0] = float(np.log(n)) * d ** 0.5
    qh = q.double().cpu().numpy()
    ref = co.attention(c, 0, qh, [0, 2], 4, d ** -0.5)
    cu.check_attention(*bd.bdlm_cache_attn_fwd(cu.to_device(bd, c), q, dev([0, 2], torch.int32), 4), ref)


def test_scores_that_grow_along_the_sequence(bd):
    # the running maximum moves in tile after tile
    c, off, q, qh = attn_case(43, [900, 600], [40, 1], 32, 8, 2, 128, 8)
    for s in range(2):
        for j, p in enumerate(c["table"][s][:co.pages_of(c["lens"][s], 32)]):
            c["ks"][0, p] *= 1 + j
    ref = co.attention(c, 0, qh, off, 8, 128 ** -0.5)
    cu.check_attention(*bd.bdlm_cache_attn_fwd(cu.to_device(bd, c), q, dev(off, torch.int32), 8), ref)


def test_malformed_rows_leave_the_outputs(bd):
    c, off, q, _ = attn_case(47, [40, 30], [4, 4], 16, 4, 2, 64, 4)
    ws = torch.empty(bd.bdlm_cache_attn_fwd_workspace_bytes(8, 4, 2, 64, 2), dtype=torch.uint8, device="cuda")
    for what, lens, cu_rows in (("order", [40, 30], [0, 5, 4]), ("total", [40, 30], [0, 4, 9]), ("start", [40, 30], [1, 4, 8]),
                                ("short", [40, 3], [0, 4, 8]), ("negative", [40, -1], [0, 8, 8]), ("long", [49, 30], [0, 4, 8])):
        cache = cu.to_device(bd, {**c, "lens": np.array(lens)})
        out, lse = torch.full_like(q, 5.0), torch.full((4, 8), 5.0, device="cuda")
        bd.bdlm_cache_attn_fwd(cache, q, dev(cu_rows, torch.int32), 4, out=out, lse=lse, workspace=ws)
        assert bd.bdlm_read_error(ws) == 6, what
        assert bool((out == 5).all()) and bool((lse == 5).all()), what
    bd.bdlm_cache_attn_fwd(cu.to_device(bd, c), q, dev(off, torch.int32), 4, out=out, lse=lse, workspace=ws)
    assert bd.bdlm_read_error(ws) == 0
    with pytest.raises(bd.BDLMError):
        bd.bdlm_cache_attn_fwd(cu.to_device(bd, c), q, dev([0, 9, 8], torch.int32), 4, check=True)


def test_a_bad_page_turns_its_sequence_into_nan(bd):
    c, off, q, qh = attn_case(53, [300, 200, 100], [4, 40, 2], 16, 4, 2, 64, 40)
    ref = co.attention(c, 0, qh, off, 40, 0.125)
    ws = torch.empty(bd.bdlm_cache_attn_fwd_workspace_bytes(46, 4, 2, 64, 3), dtype=torch.uint8, device="cuda")
    for bad in (-1, 10 ** 9, c["k"].shape[1]):
        table = c["table"].copy()
        table[1, 7] = bad  # positions 112..127 of the second sequence
        o, lse = bd.bdlm_cache_attn_fwd(cu.to_device(bd, {**c, "table": table}), q, dev(off, torch.int32), 40, workspace=ws)
        assert bd.bdlm_read_error(ws) == 6
        want = [x.copy() for x in ref]
        want[0][4:44], want[1][:, 4:44] = np.nan, np.nan
        cu.check_attention(o, lse, want)


def test_attention_is_the_same_every_time_and_wherever_pages_lie(bd):
    c, off, q, _ = attn_case(59, [5000, 77, 1300], [32, 7, 1], 16, 8, 2, 128, 32)
    cache = cu.to_device(bd, c)
    a = bd.bdlm_cache_attn_fwd(cache, q, dev(off, torch.int32), 32)
    b = bd.bdlm_cache_attn_fwd(cache, q, dev(off, torch.int32), 32)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    bd.bdlm_cache_compact(cache, check=True)
    b = bd.bdlm_cache_attn_fwd(cache, q, dev(off, torch.int32), 32)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_layers_are_apart(bd):
    c, off, q, qh = attn_case(61, [90], [3], 32, 4, 2, 64, 1, layers=3)
    cache = cu.to_device(bd, c)
    for layer in range(3):
        ref = co.attention(c, layer, qh, off, 1, 0.125)
        cu.check_attention(*bd.bdlm_cache_attn_fwd(cache, q, dev(off, torch.int32), 1, layer=layer), ref, f"layer {layer}")


# --------------------------------------------------------------------- pages
def pages_case(seed, seqs, extra=4, layers=2, page=16, hi=100, spare=40, Hk=2, d=64):
    rng = np.random.default_rng(seed)
    lens = [int(x) for x in rng.integers(0, hi, seqs)]
    return cu.make(seed, lens=lens, page=page, Hk=Hk, d=d, layers=layers, spare=spare, extra_seqs=extra,
                   max_pages=co.pages_of(2 * hi, page)), rng


@pytest.mark.parametrize("seed,seqs,page", [(0, 1, 16), (1, 7, 16), (2, 40, 32), (3, 300, 16), (4, 9000, 128)])
def test_reserve(bd, seed, seqs, page):
    c, rng = pages_case(seed, seqs, page=page, spare=8 * seqs, layers=1, Hk=1)
    cache = cu.to_device(bd, c)
    new = np.maximum(0, c["lens"] + rng.integers(-40, 60, len(c["lens"])))
    bd.bdlm_cache_reserve(cache, dev(new, torch.int32), check=True)
    assert co.reserve(c, new) == ""
    cu.check_same(cu.to_host(cache), c)


@pytest.mark.parametrize("seed,n_forks,page,d", [(0, 1, 16, 64), (1, 3, 16, 128), (2, 37, 64, 64), (3, 64, 128, 128)])
def test_fork(bd, seed, n_forks, page, d):
    c, rng = pages_case(seed, 9, extra=n_forks, page=page, spare=n_forks + 3, d=d, layers=3, hi=300)
    parents = rng.integers(0, 9, n_forks)
    children = 9 + rng.permutation(n_forks)
    lens = None if seed % 2 else np.array([rng.integers(0, c["lens"][p] + 1) for p in parents])
    cache = cu.to_device(bd, c)
    bd.bdlm_cache_fork(cache, dev(parents, torch.int32), dev(children, torch.int32),
                       None if lens is None else dev(lens, torch.int32), check=True)
    assert co.fork(c, list(parents), list(children), lens) == ""
    cu.check_same(cu.to_host(cache), c)


@pytest.mark.parametrize("seed,seqs,spare,page", [(0, 1, 1, 16), (1, 5, 60, 32), (2, 60, 300, 16), (3, 20, 0, 64), (4, 3000, 20000, 16)])
def test_compact(bd, seed, seqs, spare, page):
    c, rng = pages_case(seed, seqs, page=page, spare=spare, layers=1 if seqs > 100 else 2, Hk=1)
    if seqs > 4:
        assert co.fork(c, [1, 1, 2], [seqs, seqs + 1, seqs + 3]) in ("", "pages")  # shared pages move once
        c["lens"][3] = 0
    cache = cu.to_device(bd, c)
    live = bd.bdlm_cache_compact(cache, check=True)
    assert int(live) == co.compact(c)
    cu.check_same(cu.to_host(cache), c)
    live = bd.bdlm_cache_compact(cache, check=True)  # nothing is left to move
    assert int(live) == co.compact(c)
    cu.check_same(cu.to_host(cache), c)


def test_page_calls_that_fail_change_nothing(bd):
    c, _ = pages_case(5, 6, spare=2)
    c["lens"][:6] = np.maximum(c["lens"][:6], 1)
    for s in range(6):
        c["table"][s, :co.pages_of(c["lens"][s], 16)] = np.where(c["table"][s, :co.pages_of(c["lens"][s], 16)] < 0, 0, c["table"][s, :co.pages_of(c["lens"][s], 16)])
    ws = torch.empty(bd.bdlm_cache_pages_workspace_bytes(c["k"].shape[1], 10), dtype=torch.uint8, device="cuda")
    i32 = lambda *x: dev(x, torch.int32)
    more = c["lens"].copy()
    more[3] += 150 if more[3] + 150 <= 13 * 16 else 90
    far = c["lens"].copy()
    far[2] = 13 * 16 + 1
    neg = c["lens"].copy()
    neg[5] = -1
    every = np.full_like(c["lens"], 13 * 16)
    torn = {**c, "table": c["table"].copy()}
    torn["table"][0, 0] = c["k"].shape[1]
    runs = [
        (7, c, lambda x: bd.bdlm_cache_reserve(x, dev(more, torch.int32), workspace=ws)),
        (7, c, lambda x: bd.bdlm_cache_reserve(x, dev(every, torch.int32), workspace=ws)),
        (6, c, lambda x: bd.bdlm_cache_reserve(x, dev(far, torch.int32), workspace=ws)),
        (6, c, lambda x: bd.bdlm_cache_reserve(x, dev(neg, torch.int32), workspace=ws)),
        (6, torn, lambda x: bd.bdlm_cache_reserve(x, dev(c["lens"], torch.int32), workspace=ws)),
        (6, torn, lambda x: bd.bdlm_cache_compact(x, workspace=ws)),
        (6, c, lambda x: bd.bdlm_cache_fork(x, i32(0, 1), i32(6, 6), workspace=ws)),        # a child twice
        (6, c, lambda x: bd.bdlm_cache_fork(x, i32(0), i32(1), workspace=ws)),              # a child that holds something
        (6, c, lambda x: bd.bdlm_cache_fork(x, i32(0, 6), i32(6, 7), workspace=ws)),        # parent and child at once
        (6, c, lambda x: bd.bdlm_cache_fork(x, i32(6), i32(6), workspace=ws)),
        (6, c, lambda x: bd.bdlm_cache_fork(x, i32(0), i32(10), workspace=ws)),             # no such sequence
        (6, c, lambda x: bd.bdlm_cache_fork(x, i32(-1), i32(6), workspace=ws)),
        (6, c, lambda x: bd.bdlm_cache_fork(x, i32(0), i32(6), dev(c["lens"][:1] + 1, torch.int32), workspace=ws)),
    ]
    for i, (status, host, call) in enumerate(runs):
        cache = cu.to_device(bd, host)
        call(cache)
        assert bd.bdlm_read_error(ws) == status, i
        cu.check_same(cu.to_host(cache), host, f"run {i}")
    with pytest.raises(bd.BDLMError, match="NO_PAGES"):
        bd.bdlm_cache_reserve(cu.to_device(bd, c), dev(every, torch.int32), check=True)


def test_growing_inside_a_shared_page_is_refused(bd):
    c = cu.make(71, lens=[40, 0], page=16, Hk=1, d=64, spare=4, max_pages=8)
    cache = cu.to_device(bd, c)
    bd.bdlm_cache_fork(cache, dev([0], torch.int32), dev([1], torch.int32), check=True)
    cache.lens[1] = 20  # inside page 1, which both read
    with pytest.raises(bd.BDLMError):
        bd.bdlm_cache_reserve(cache, dev([40, 21], torch.int32), check=True)
    bd.bdlm_cache_reserve(cache, dev([40, 16], torch.int32), check=True)  # shrinking to the page's end is fine
    bd.bdlm_cache_reserve(cache, dev([40, 30], torch.int32), check=True)
    t = cache.table.cpu()
    assert t[1, 0] == t[0, 0] and t[1, 1] != t[0, 1]


# ------------------------------------------------------------------ together
def test_answering_block_by_block(bd):
    """Prompts, denoising steps, candidates, endings and a compaction, as a program would run them; every
    attention is compared with the oracle over a host copy that follows along."""
    from block_diffusion_lm_bdlm_gb300.decode import BlockDecoder

    H, Hk, d, page, B, layers = 8, 2, 64, 16, 8, 2
    cache = bd.PageCache.empty(layers, 60, page, Hk, d, 6, 12)
    host = cu.to_host(cache)
    dec = BlockDecoder(cache, B)
    rng = np.random.default_rng(73)

    def step(rows, times, layer_check=(0, 1)):
        cu_rows = dec.begin(dev(rows, torch.int32), check=True)
        assert co.reserve(host, host["lens"] + rows) == ""
        off = cu.offsets(rows)
        assert np.array_equal(cu_rows.cpu().numpy(), off)
        T = int(off[-1])
        for _ in range(times):
            for layer in range(layers):
                (q, qh), (k, kh), (v, vh) = rows_of(rng, T, H, d), rows_of(rng, T, Hk, d), rows_of(rng, T, Hk, d)
                o, lse = dec.attend(layer, q, k, v)
                co.write(host, layer, kh, vh, off)
                cu.check_attention(o, lse, co.attention(host, layer, qh, off, B, d ** -0.5))
        cu.check_same(cu.to_host(cache), host)

    step(np.array([24, 40, 16, 0, 0, 0]), 1)       # prompts
    step(np.array([8, 8, 8, 0, 0, 0]), 3)          # a block, three denoising steps
    step(np.array([8, 0, 8, 0, 0, 0]), 1)
    dec.rewind()                                   # a block that is given up
    host["lens"] = np.array([32, 48, 24, 0, 0, 0])
    dec.branch(dev([0, 2, 2], torch.int32), dev([3, 4, 5], torch.int32), check=True)
    assert co.fork(host, [0, 2, 2], [3, 4, 5]) == ""
    step(np.array([8, 8, 8, 8, 8, 8]), 2)          # parents and candidates go their own ways
    dec.end(dev([0, 4], torch.int32))
    host["lens"][[0, 4]] = 0
    live = bd.bdlm_cache_compact(cache, check=True)
    assert int(live) == co.compact(host)
    step(np.array([13, 8, 0, 8, 0, 1]), 1)         # slot 0 is used again
    cu.check_same(cu.to_host(cache), host)


def test_a_step_captured_in_a_cuda_graph(bd):
    # reserve, write and attention captured once, replayed for block after block: the lengths live on the device
    H, Hk, d, page, B = 4, 2, 128, 32, 16
    c = cu.make(79, lens=[33, 300], page=page, Hk=Hk, d=d, spare=30, max_pages=16)
    cache = cu.to_device(bd, c)
    T = 2 * B
    q = torch.zeros(T, H, d, dtype=torch.bfloat16, device="cuda")
    k, v = torch.zeros(T, Hk, d, dtype=torch.bfloat16, device="cuda"), torch.zeros(T, Hk, d, dtype=torch.bfloat16, device="cuda")
    off = dev([0, B, T], torch.int32)
    new = cache.lens.clone()

    def step():
        torch.add(cache.lens, B, out=new)
        bd.bdlm_cache_reserve(cache, new)
        bd.bdlm_cache_write(cache, k, v, off)
        return bd.bdlm_cache_attn_fwd(cache, q, off, B)

    keep = [x.clone() for x in (cache.k.view(torch.uint8), cache.v.view(torch.uint8), cache.k_scale, cache.v_scale, cache.table, cache.lens)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    for x, y in zip((cache.k.view(torch.uint8), cache.v.view(torch.uint8), cache.k_scale, cache.v_scale, cache.table, cache.lens), keep):
        x.copy_(y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = step()
    rng = np.random.default_rng(83)
    for i in range(3):
        (q1, qh), (k1, kh), (v1, vh) = rows_of(rng, T, H, d), rows_of(rng, T, Hk, d), rows_of(rng, T, Hk, d)
        q.copy_(q1), k.copy_(k1), v.copy_(v1)
        graph.replay()
        assert co.reserve(c, c["lens"] + B) == ""
        co.write(c, 0, kh, vh, [0, B, T])
        cu.check_same(cu.to_host(cache), c, f"replay {i}")
        cu.check_attention(o, lse, co.attention(c, 0, qh, [0, B, T], B, d ** -0.5), f"replay {i}")


def test_another_stream(bd):
    c, off, q, qh = attn_case(89, [700, 60], [16, 16], 16, 4, 2, 64, 16)
    cache = cu.to_device(bd, c)
    ref = co.attention(c, 0, qh, off, 16, 0.125)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for stream in (s, s.cuda_stream):
        o, lse = bd.bdlm_cache_attn_fwd(cache, q, dev(off, torch.int32), 16, stream=stream)
        s.synchronize()
        cu.check_attention(o, lse, ref)
    assert bd.bdlm_last_launch_count() >= 1


def test_the_binding_refuses(bd):
    c, off, q, _ = attn_case(97, [40], [4], 16, 4, 2, 64, 4)
    cache = cu.to_device(bd, c)
    o32 = dev(off, torch.int32)
    k = torch.zeros(4, 2, 64, dtype=torch.bfloat16, device="cuda")
    bad = [
        lambda: bd.bdlm_cache_attn_fwd(cache, q.float(), o32, 4),
        lambda: bd.bdlm_cache_attn_fwd(cache, q[:, :, :32].contiguous(), o32, 4),
        lambda: bd.bdlm_cache_attn_fwd(cache, q.transpose(0, 1), o32, 4),
        lambda: bd.bdlm_cache_attn_fwd(cache, q, o32.long(), 4),
        lambda: bd.bdlm_cache_attn_fwd(cache, q, o32[:1], 4),
        lambda: bd.bdlm_cache_attn_fwd(cache, q, o32.cpu(), 4),
        lambda: bd.bdlm_cache_attn_fwd(cache, q, o32, 4, layer=1),
        lambda: bd.bdlm_cache_attn_fwd(cache, q, o32, 4, q_pos=o32),
        lambda: bd.bdlm_cache_attn_fwd(cache, q, o32, 4, out=q.half()),
        lambda: bd.bdlm_cache_attn_fwd(cache, q, o32, 4, lse=torch.zeros(4, 4, device="cuda").double()),
        lambda: bd.bdlm_cache_attn_fwd(cache, q, o32, 4, workspace=torch.empty(1 << 20, device="cuda")),
        lambda: bd.bdlm_cache_write(cache, k, k[:3], o32),
        lambda: bd.bdlm_cache_write(cache, k[:, :1].contiguous(), k[:, :1].contiguous(), o32),
        lambda: bd.bdlm_cache_reserve(cache, o32),
        lambda: bd.bdlm_cache_fork(cache, o32[:1], o32),
        lambda: bd.PageCache(cache.k, cache.v, cache.k_scale, cache.v_scale, cache.table, cache.lens.long()),
        lambda: bd.PageCache(cache.k, cache.v, cache.k_scale[:, :-1], cache.v_scale, cache.table, cache.lens),
        lambda: bd.PageCache.empty(1, 4, 48, 1, 64, 1, 1),
        lambda: bd.PageCache.empty(1, 4, 16, 1, 96, 1, 1),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            pytest.fail(f"call {i} was taken")
    for f in (lambda: bd.bdlm_cache_attn_fwd(cache, q[:, :3].contiguous(), o32, 4), lambda: bd.bdlm_cache_attn_fwd(cache, q, o32, 0),
              lambda: bd.bdlm_cache_attn_fwd(cache, q, o32, 4, workspace=torch.empty(128, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(bd.BDLMError):
            f()
