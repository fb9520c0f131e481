"""The cache oracle pinned on the CPU: codes against torch's e4m3 conversion, scales against their
definition, attention against the BDLM oracle, the page calls against their invariants; and the tests' own
error bound against a planted mistake."""
import numpy as np
import pytest
import torch

import oracle
from oracle import cache_oracle as co

import cache_util as cu


def test_codes_are_e4m3():
    v = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(np.isnan(v), np.isnan(co.VALUES))
    assert np.array_equal(v[~np.isnan(v)], co.VALUES[~np.isnan(v)])
    rng = np.random.default_rng(0)
    x = np.concatenate([rng.uniform(-448, 448, 4000), rng.standard_normal(4000) * 2.0 ** rng.integers(-14, 8, 4000)])
    mid = (co.VALUES[:126] + co.VALUES[1:127]) / 2  # ties
    x = np.clip(np.concatenate([x, mid, -mid, [0.0, -0.0, 448.0]]), -448, 448).astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(co.encode(x.astype(np.float64)), want)
    assert list(co.encode([np.inf, -np.inf, np.nan])) == [127, 127, 127]


@pytest.mark.parametrize("amax,scale", [(0.0, 1.0), (448.0, 1.0), (448.5, 2.0), (224.0, 0.5), (224.1, 1.0), (1.75, 2.0 ** -8),
                                        (1.76, 2.0 ** -7), (1e-45, 2.0 ** -126), (3.3e38, 2.0 ** 120)])
def test_scale(amax, scale):
    assert co.pow2_scale(amax) == scale


def test_attention_agrees_with_the_clean_half_of_the_bdlm_oracle():
    # clean rows of a BDLM sequence see the clean blocks <= their own: the cache's mask, here with ragged last blocks
    n, B, H, Hk, d, page = 53, 8, 4, 2, 64, 16
    c = cu.make(1, lens=[n], page=page, Hk=Hk, d=d)
    rng = np.random.default_rng(2)
    q = rng.standard_normal((n, H, d))
    o, lse, *_ = co.attention(c, 0, q, [0, n], B, d ** -0.5)
    ids = c["table"][0, :co.pages_of(n, page)]
    flat = lambda x: np.stack([(co.VALUES[c[x][0, ids, h]] * c[x + "s"][0, ids, h][:, None, None]).reshape(-1, d)[:n] for h in range(Hk)], 1)
    k, v = flat("k"), flat("v")
    ref = oracle.bdlm_attention(np.concatenate([q, q]), np.concatenate([k, k]), np.concatenate([v, v]), B, d ** -0.5)
    assert np.allclose(o, ref["o"][:n], atol=1e-12) and np.allclose(lse, ref["lse"][:, :n], atol=1e-12)


def test_a_row_without_keys_is_empty():
    c = cu.make(3, lens=[0, 5], page=16, Hk=1, d=64)
    o, lse, *_ = co.attention(c, 0, np.ones((3, 2, 64)), [0, 2, 3], 4, 0.1, q_pos=[0, 2])
    assert np.all(o[:2] == 0) and np.all(np.isneginf(lse[:, :2])) and np.all(np.isfinite(lse[:, 2]))


def test_writing_twice_changes_nothing_and_keeps_values():
    c = cu.make(4, lens=[40, 7], page=16, Hk=2, d=64, max_pages=8)
    assert co.reserve(c, [49, 12]) == ""
    rng = np.random.default_rng(5)
    new = rng.standard_normal((14, 2, 64)) * 3
    before = {x: c[x].copy() for x in ("k", "v", "ks", "vs")}
    co.write(c, 0, new, new, [0, 9, 14])
    once = {x: c[x].copy() for x in ("k", "v", "ks", "vs")}
    co.write(c, 0, new, new, [0, 9, 14])
    assert all(np.array_equal(once[x], c[x]) for x in once)
    pid = c["table"][0, 2]
    was = co.VALUES[before["k"][0, pid, 0, :8]] * before["ks"][0, pid, 0]
    now = co.VALUES[c["k"][0, pid, 0, :8]] * c["ks"][0, pid, 0]
    assert np.all(np.abs(was - now) <= 2.0 ** -10 * c["ks"][0, pid, 0])  # half a subnormal step of the new scale


def test_reserve_fork_compact_keep_what_sequences_hold():
    c = cu.make(6, lens=[37, 64, 5], page=16, Hk=1, d=64, layers=2, spare=9, extra_seqs=3, max_pages=6)
    hold = lambda s: [(c["k"][:, p], c["ks"][:, p]) for p in c["table"][s, :co.pages_of(c["lens"][s], 16)]]
    old = [hold(s) for s in range(3)]
    assert co.fork(c, [0, 0, 1], [3, 4, 5]) == ""
    assert co.reserve(c, [40, 64, 5, 60, 37, 64]) == ""
    c["lens"][1] = 0
    live = co.compact(c)
    assert live == (co.live_pages(c) > 0).sum() and c["table"][0, :3].max() < live
    for s in (0, 2):
        for (k0, s0), (k1, s1) in zip(old[s], hold(s)):
            assert np.array_equal(k0, k1) and np.array_equal(s0, s1)
    assert np.array_equal(c["table"][4, :2], c["table"][0, :2]) and c["table"][4, 2] != c["table"][0, 2]
    assert co.fork(c, [0], [0]) == "children" and co.fork(c, [0, 0], [1, 1]) == "children"
    c["lens"][3] = 20  # inside page 1, which sequence 0 reads too
    assert co.reserve(c, [40, 0, 5, 21, 37, 64]) == "shared"


def test_the_bound_sees_a_mistake():
    c = cu.make(7, lens=[300], page=32, Hk=2, d=64)
    q = np.random.default_rng(8).standard_normal((3, 4, 64))
    ref = co.attention(c, 0, q, [0, 3], 1, 0.125)
    good = torch.from_numpy(ref[0]).bfloat16(), torch.from_numpy(ref[1]).float()
    cu.check_attention(*good, ref)
    wrong = co.attention({**c, "lens": np.array([299])}, 0, q, [0, 3], 1, 0.125, q_pos=[297])
    with pytest.raises(AssertionError):
        cu.check_attention(torch.from_numpy(wrong[0]).bfloat16(), torch.from_numpy(wrong[1]).float(), ref)
