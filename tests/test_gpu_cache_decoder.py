"""BlockDecoder where a program leaves the plain order of prompt, blocks and endings: numbers that name no sequence,
blocks that are given up, sequences that end or branch between two steps of a block, calls without rows."""
import numpy as np
import pytest
import torch

from oracle import cache_oracle as co

import cache_util as cu
from test_gpu_cache import bd, dev, rows_of  # noqa: F401  (bd is a fixture)

pytestmark = pytest.mark.gpu


def decoder(bd, seed, lens, *, page=16, Hk=2, d=64, block=8, spare=20, extra_seqs=2, layers=1):
    """(decoder, its cache, a host copy of it)"""
    from block_diffusion_lm_bdlm_gb300.decode import BlockDecoder

    c = cu.make(seed, lens=lens, page=page, Hk=Hk, d=d, spare=spare, extra_seqs=extra_seqs, layers=layers, max_pages=8)
    cache = cu.to_device(bd, c)
    return BlockDecoder(cache, block), cache, c


def i32(*x):
    return dev(list(x), torch.int32)


def test_ending_numbers_that_name_no_sequence(bd):
    dec, cache, c = decoder(bd, 401, [20, 9, 33])
    for seqs in (i32(5, 99, -6, 2 ** 31 - 1), i32(), dev([2 ** 40], torch.int64)):
        dec.end(seqs)
        cu.check_same(cu.to_host(cache), c)
    dec.end(i32(1, 77, 1))
    dec.end(torch.tensor([-3]))  # from the end: sequence 2 of five
    c["lens"][1:3] = 0
    cu.check_same(cu.to_host(cache), c)
    for seqs in (torch.tensor([True, False, False, False, False]), torch.tensor([0.0])):
        with pytest.raises(ValueError):
            dec.end(seqs)
    cu.check_same(cu.to_host(cache), c)


def test_rewind_leaves_endings_and_candidates_as_they_are(bd):
    # begin, end one sequence, branch into its pages and its place, compact, rewind: what ended stays ended, what
    # branched stays, and only the others lose the block's rows
    dec, cache, c = decoder(bd, 409, [24, 40, 16, 30])
    dec.begin(i32(8, 8, 0, 8, 0, 0), check=True)
    assert co.reserve(c, c["lens"] + [8, 8, 0, 8, 0, 0]) == ""
    dec.end(i32(1))
    c["lens"][1] = 0
    dec.branch(i32(2, 0), i32(1, 4), check=True)  # 1 again, now 16 positions; 4 holds sequence 0's 32
    assert co.fork(c, [2, 0], [1, 4]) == ""
    assert int(bd.bdlm_cache_compact(cache, check=True)) == co.compact(c)
    cu.check_same(cu.to_host(cache), c)
    dec.rewind()
    c["lens"] = np.array([24, 16, 16, 30, 32, 0])
    cu.check_same(cu.to_host(cache), c)
    dec.rewind()  # there is nothing left to drop
    cu.check_same(cu.to_host(cache), c)


@pytest.mark.parametrize("direct", [False, True])
def test_rewind_passes_over_a_child_as_long_as_the_sequence_that_ended_in_its_place(bd, direct):
    dec, cache, c = decoder(bd, 419, [24, 24])
    dec.begin(i32(8, 8, 0, 0), check=True)
    assert co.reserve(c, c["lens"] + [8, 8, 0, 0]) == ""
    if direct:
        cache.lens[0] = 0
    else:
        dec.end(i32(0))
    c["lens"][0] = 0
    dec.branch(i32(1), i32(0), check=True)
    assert co.fork(c, [1], [0]) == ""
    dec.rewind()
    c["lens"] = np.array([32, 24, 0, 0])
    cu.check_same(cu.to_host(cache), c)


def test_attending_after_rewind_touches_nothing(bd):
    dec, cache, c = decoder(bd, 421, [24, 33])
    rng = np.random.default_rng(1)
    (q, _), (k, _), (v, _) = rows_of(rng, 16, 4, 64), rows_of(rng, 16, 2, 64), rows_of(rng, 16, 2, 64)
    for again in (False, True):  # before the first begin, and after rewind
        out, lse = torch.full_like(q, 5.0), torch.full((4, 16), 5.0, device="cuda")
        dec.attend(0, q, k, v, out=out, lse=lse)
        assert bool((out == 5).all()) and bool((lse == 5).all())
        got = cu.to_host(cache)
        cu.check_same({**got, "table": c["table"]}, c)
        if again:
            with pytest.raises(RuntimeError, match="begin"):
                dec.attend(0, q, k, v, out=out, lse=lse, check=True)
        else:
            assert dec.begin(i32(8, 8, 0, 0), check=True).tolist() == [0, 8, 16, 16, 16]
            dec.rewind()
            assert dec.cu_rows.tolist() == [0, 8, 16, 16, 16]  # what begin has returned is the program's to read


@pytest.mark.parametrize("direct", [False, True])
def test_a_sequence_that_ends_between_two_steps(bd, direct):
    # its rows are not written and see nothing; the others go on in their places of q, k and v, also behind a rewind
    dec, cache, c = decoder(bd, 431, [24, 40, 16], Hk=2, d=64, block=8)
    rows = np.array([8, 8, 8, 0, 0])
    off = cu.offsets(rows)
    rng = np.random.default_rng(2)

    def step(dead):
        (q, qh), (k, kh), (v, vh) = rows_of(rng, 24, 4, 64), rows_of(rng, 24, 2, 64), rows_of(rng, 24, 2, 64)
        o, lse = dec.attend(0, q, k, v)
        if not dead:
            co.write(c, 0, kh, vh, off)
            cu.check_attention(o, lse, co.attention(c, 0, qh, off, 8, 0.125))
            return
        co.write(c, 0, np.delete(kh, slice(8, 16), 0), np.delete(vh, slice(8, 16), 0), [0, 8, 8, 16, 16, 16])
        cu.check_attention(o, lse, co.attention(c, 0, qh, off, 8, 0.125, q_pos=[24, 40, 16, 0, 0]))
        assert bool((o[8:16] == 0).all()) and bool(torch.isneginf(lse[:, 8:16]).all())
        cu.check_same(cu.to_host(cache), c)

    dec.begin(dev(rows, torch.int32), check=True)
    assert co.reserve(c, c["lens"] + rows) == ""
    step(False)
    if direct:
        cache.lens[1] = 0
    else:
        dec.end(i32(1))
    c["lens"][1] = 0
    step(True)
    step(True)
    dec.rewind()
    c["lens"] = np.array([24, 0, 16, 0, 0])
    cu.check_same(cu.to_host(cache), c)


def test_checked_attending_raises_for_offsets_that_do_not_fit(bd):
    dec, _, _ = decoder(bd, 433, [24, 33])
    dec.begin(i32(8, 8, 0, 0), check=True)
    q, k = torch.ones(15, 4, 64, dtype=torch.bfloat16, device="cuda"), torch.ones(15, 2, 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(bd.BDLMError):
        dec.attend(0, q, k, k, check=True)


@pytest.mark.parametrize("page,over", [(16, True), (64, False)])
def test_branching_between_two_steps(bd, page, over):
    # 24 positions and a block of 8: with 16-row pages parent and child share rows 16 .. 31 and the block is over; with
    # 64-row pages the child has a copy of them and the parent goes on
    dec, cache, c = decoder(bd, 439, [24, 40], page=page)
    rng = np.random.default_rng(3)
    off = [0, 8, 16, 16, 16]

    def step(over):
        (q, qh), (k, kh), (v, vh) = rows_of(rng, 16, 4, 64), rows_of(rng, 16, 2, 64), rows_of(rng, 16, 2, 64)
        out, lse = torch.full_like(q, 5.0), torch.full((4, 16), 5.0, device="cuda")
        dec.attend(0, q, k, v, out=out, lse=lse)
        if over:
            assert bool((out == 5).all()) and bool((lse == 5).all())
        else:
            co.write(c, 0, kh, vh, off)
            cu.check_attention(out, lse, co.attention(c, 0, qh, off, 8, 0.125, q_pos=[24, 40, 0, 0]))
        cu.check_same(cu.to_host(cache), c)

    dec.begin(i32(8, 8, 0, 0), check=True)
    assert co.reserve(c, c["lens"] + [8, 8, 0, 0]) == ""
    step(False)
    dec.branch(i32(0), i32(1))  # refused: child 1 is not empty; the block goes on
    step(False)
    dec.branch(i32(0), i32(2), check=True)
    assert co.fork(c, [0], [2]) == ""
    step(over)
    dec.begin(i32(0, 8, 8, 0), check=True)
    assert co.reserve(c, c["lens"] + [0, 8, 8, 0]) == ""
    assert dec.cu_rows.tolist() == [0, 0, 8, 16, 16]


def test_branching_what_takes_no_part_in_the_block(bd):
    dec, cache, c = decoder(bd, 443, [24, 40])
    rng = np.random.default_rng(4)
    off = [0, 8, 8, 8, 8]
    dec.begin(i32(8, 0, 0, 0), check=True)
    assert co.reserve(c, c["lens"] + [8, 0, 0, 0]) == ""
    dec.branch(i32(1), i32(3), check=True)
    assert co.fork(c, [1], [3]) == ""
    (q, qh), (k, kh), (v, vh) = rows_of(rng, 8, 4, 64), rows_of(rng, 8, 2, 64), rows_of(rng, 8, 2, 64)
    o, lse = dec.attend(0, q, k, v, check=True)
    co.write(c, 0, kh, vh, off)
    cu.check_attention(o, lse, co.attention(c, 0, qh, off, 8, 0.125))
    cu.check_same(cu.to_host(cache), c)


def test_branching_into_the_place_of_a_sequence_with_rows(bd):
    dec, cache, c = decoder(bd, 449, [24, 40, 20])
    dec.begin(i32(8, 8, 0, 0, 0), check=True)
    assert co.reserve(c, c["lens"] + [8, 8, 0, 0, 0]) == ""
    dec.end(i32(0))
    c["lens"][0] = 0
    dec.branch(i32(2), i32(0), check=True)
    assert co.fork(c, [2], [0]) == ""
    q, k = torch.ones(16, 4, 64, dtype=torch.bfloat16, device="cuda"), torch.ones(16, 2, 64, dtype=torch.bfloat16, device="cuda")
    dec.attend(0, q, k, k)  # sequence 0's rows are not the child's
    cu.check_same(cu.to_host(cache), c)


@pytest.mark.parametrize("bad", ["room", "negative", "long", "type"])
def test_a_block_that_is_refused_has_no_rows(bd, bad):
    dec, cache, c = decoder(bd, 457, [24, 40], spare=3)
    q, k = torch.ones(16, 4, 64, dtype=torch.bfloat16, device="cuda"), torch.ones(16, 2, 64, dtype=torch.bfloat16, device="cuda")
    dec.begin(i32(8, 8, 0, 0), check=True)
    assert co.reserve(c, c["lens"] + [8, 8, 0, 0]) == ""
    rows = {"room": i32(64, 64, 0, 0), "negative": i32(8, -3, 0, 0), "long": i32(2 ** 31 - 1, 0, 0, 0),
            "type": dev([8, 8, 0, 0], torch.int64)}[bad]
    with pytest.raises(ValueError if bad == "type" else bd.BDLMError):
        dec.begin(rows, check=True)
    assert dec.cu_rows.tolist() == [0] * 5
    dec.attend(0, q, k, k)  # not the block before's rows
    dec.rewind()
    cu.check_same(cu.to_host(cache), c)
    if bad != "type":
        assert dec.begin(rows).tolist() == [0] * 5
        cu.check_same(cu.to_host(cache), c)
    assert dec.begin(i32(8, 0, 0, 0), check=True).tolist() == [0, 8, 8, 8, 8]


def test_a_step_in_which_no_sequence_takes_part(bd):
    dec, cache, c = decoder(bd, 461, [24, 40])
    q, k = torch.ones(0, 4, 64, dtype=torch.bfloat16, device="cuda"), torch.ones(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    dec.begin(i32(0, 0, 0, 0), check=True)
    for check in (False, True):
        o, lse = dec.attend(0, q, k, k, check=check)
        assert o.shape == (0, 4, 64) and lse.shape == (4, 0)
    ws = torch.full((1 << 20,), 255, dtype=torch.uint8, device="cuda")
    none, some = i32(0, 0, 0, 0, 0), i32(0, 0, 8, 8, 8)
    for cu_rows, status in ((some, 6), (none, 0)):
        bd.bdlm_cache_write(cache, k, k, cu_rows, workspace=ws)
        assert bd.bdlm_read_error(ws) == status
        ws.fill_(255)
        bd.bdlm_cache_attn_fwd(cache, q, cu_rows, 8, workspace=ws)
        assert bd.bdlm_read_error(ws) == status
        if status:
            for call in (lambda: bd.bdlm_cache_write(cache, k, k, cu_rows, check=True),
                         lambda: bd.bdlm_cache_attn_fwd(cache, q, cu_rows, 8, check=True)):
                with pytest.raises(bd.BDLMError):
                    call()
    with pytest.raises(bd.BDLMError):
        bd.bdlm_cache_attn_fwd(cache, q[:, :3].contiguous(), none, 8)
    with pytest.raises(ValueError):
        bd.bdlm_cache_write(cache, k, k[:, :1].contiguous(), none)
    cu.check_same(cu.to_host(cache), c)


def test_branching_nothing(bd):
    dec, cache, c = decoder(bd, 463, [24, 40])
    dec.branch(i32(), i32(), check=True)
    ws = torch.full((4096,), 255, dtype=torch.uint8, device="cuda")
    bd.bdlm_cache_fork(cache, i32(), i32(), i32(), workspace=ws)
    assert bd.bdlm_read_error(ws) == 0
    with pytest.raises(ValueError):
        bd.bdlm_cache_fork(cache, i32(), i32(1))
    cu.check_same(cu.to_host(cache), c)


def test_blocks_from_captured_graphs(bd):
    # one graph gives every sequence a block, one attends, one gives the block up, one ends a sequence: replayed in any
    # order, with eager calls between them
    dec, cache, c = decoder(bd, 467, [24, 40], spare=30)
    rows, gone = i32(8, 8, 0, 0), i32(1)
    q, k, v, o = (torch.zeros(16, n, 64, dtype=torch.bfloat16, device="cuda") for n in (4, 2, 2, 4))
    lse = torch.zeros(4, 16, device="cuda")
    keep = [x.clone() for x in (cache.k.view(torch.uint8), cache.v.view(torch.uint8), cache.k_scale, cache.v_scale, cache.table, cache.lens)]
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        dec.begin(rows), dec.attend(0, q, k, v), dec.rewind(), dec.end(gone)
    torch.cuda.synchronize()
    for x, y in zip((cache.k.view(torch.uint8), cache.v.view(torch.uint8), cache.k_scale, cache.v_scale, cache.table, cache.lens), keep):
        x.copy_(y)
    graphs = []
    for f in (lambda: dec.begin(rows), lambda: dec.attend(0, q, k, v, out=o, lse=lse), dec.rewind, lambda: dec.end(gone)):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            f()
    begin, attend, rewind, end = (g.replay for g in graphs)
    rng = np.random.default_rng(5)
    off, pos = [0, 8, 16, 16, 16], None

    def step(alone=False):
        (q1, qh), (k1, kh), (v1, vh) = rows_of(rng, 16, 4, 64), rows_of(rng, 16, 2, 64), rows_of(rng, 16, 2, 64)
        q.copy_(q1), k.copy_(k1), v.copy_(v1)
        attend()
        if alone:
            co.write(c, 0, kh[:8], vh[:8], [0, 8, 8, 8, 8])
        else:
            co.write(c, 0, kh, vh, off)
        cu.check_attention(o, lse, co.attention(c, 0, qh, off, 8, 0.125, q_pos=pos))
        cu.check_same(cu.to_host(cache), c)

    for give_up in (False, True, False):
        pos = list(c["lens"])
        begin()
        assert co.reserve(c, c["lens"] + [8, 8, 0, 0]) == ""
        step(), step()
        if give_up:
            rewind()
            c["lens"] = np.array(pos)
            o.fill_(5.0)
            attend()
            assert bool((o == 5).all())
            cu.check_same(cu.to_host(cache), c)
    end()
    c["lens"][1] = 0
    step(alone=True)
    pos = list(c["lens"])
    dec.begin(rows, check=True)  # sequence 1 anew
    assert co.reserve(c, c["lens"] + [8, 8, 0, 0]) == ""
    step()
