"""Helpers of the cache tests: random caches on the host and on the device, and
the error bounds of the attention over them.

The bounds count roundings. With u(t) = finfo(t).eps / 2 the half step of a type:
  scores   products of e4m3 keys with bf16 queries, summed in fp32. The worst case of d <= 128 sequential roundings by
           truncation is 128 * 2^-23 = 2^-16 of S1 = max_j scale sum |q k|; the queries may be held as two terms of 8 bits
           under a power-of-two scale per row, off by at most 2^-10 / 224 < 2^-17 of the row's largest entry each, which
           adds at most d * 2^-17 * max|q| * max|k| * scale <= 2^-17 * S2, where S2 = scale * d * max|q| * max|k|. With
           the scales (2^-24 each) and the exponent's own roundings both stay below ds = 2^-15 S1 + 2^-16 S2.
  lse      moves by at most ds, plus the logarithm's and the sum's roundings (2^-20 of 1 + |lse|).
  weights  held in fp16 (2^-11) or fp32 and moved by ds both above and below the fraction bar: o moves by at most
           (2^-11 + 2^-12 + 2 ds) A, A = sum p |v| (the 2^-12 for exponentials, values scaled in fp16 and fp32 sums).
  o        rounded once to its own type.
"""
import numpy as np
import torch

from oracle import cache_oracle as co


def make(seed, *, lens, page, Hk, d, layers=1, spare=3, max_pages=None, extra_seqs=0, k_std=1.0, v_std=1.0, page_spread=1.0):
    """A host cache whose sequences hold `lens` positions of random values in
    randomly placed pages; unused rows and pages hold random codes, NaN among them."""
    rng = np.random.default_rng(seed)
    need = [co.pages_of(n, page) for n in lens]
    total = sum(need) + spare
    ids = rng.permutation(total)
    c = {}
    for name, std in (("k", k_std), ("v", v_std)):
        c[name] = rng.integers(0, 256, (layers, total, Hk, page, d), dtype=np.uint8)  # stale rows may be NaN
        c[name + "s"] = np.exp2(rng.integers(-3, 4, (layers, total, Hk)).astype(np.float64))
    cap = max_pages or max(need + [1])
    c["table"] = np.full((len(lens) + extra_seqs, cap), -7, dtype=np.int64)
    at = 0
    for s, (n, m) in enumerate(zip(lens, need)):
        c["table"][s, :m] = ids[at:at + m]
        for j in range(m):
            rows = min(page, n - j * page)
            for name, std in (("k", k_std), ("v", v_std)):
                x = rng.standard_normal((layers, Hk, rows, d)) * std * np.exp2(page_spread * rng.standard_normal((layers, Hk, 1, 1)))
                for la in range(layers):
                    for h in range(Hk):
                        sc = co.pow2_scale(float(np.abs(x[la, h]).max()))
                        c[name][la, ids[at + j], h, :rows] = co.encode(x[la, h] / sc)
                        c[name + "s"][la, ids[at + j], h] = sc
        at += m
    c["lens"] = np.array(list(lens) + [0] * extra_seqs, dtype=np.int64)
    return c


def to_device(bd, c, device="cuda"):
    f8 = lambda x: torch.from_numpy(x.copy()).to(device).view(torch.float8_e4m3fn)
    f32 = lambda x: torch.from_numpy(x.astype(np.float32)).to(device)
    i32 = lambda x: torch.from_numpy(x.astype(np.int32)).to(device)
    return bd.PageCache(f8(c["k"]), f8(c["v"]), f32(c["ks"]), f32(c["vs"]), i32(c["table"]), i32(c["lens"]))


def to_host(cache):
    return {"k": cache.k.view(torch.uint8).cpu().numpy(), "v": cache.v.view(torch.uint8).cpu().numpy(),
            "ks": cache.k_scale.double().cpu().numpy(), "vs": cache.v_scale.double().cpu().numpy(),
            "table": cache.table.cpu().numpy().astype(np.int64), "lens": cache.lens.cpu().numpy().astype(np.int64)}


def same_codes(a, b):
    """Equal codes; every NaN code counts as the same."""
    return bool(np.all((a == b) | (((a & 127) == 127) & ((b & 127) == 127))))


def check_same(got, want, what=""):
    for name in ("table", "lens", "ks", "vs"):
        assert np.array_equal(got[name], want[name]), f"{what}: {name} differs"
    for name in "kv":
        assert same_codes(got[name], want[name]), f"{what}: codes of {name} differ"


def offsets(rows):
    return np.concatenate([[0], np.cumsum(rows)]).astype(np.int64)


def check_attention(got_o, got_lse, ref, what=""):
    """got_o [T,H,d] tensor (bf16 or fp32), got_lse [H,T]; ref from cache_oracle.attention."""
    o, lse, A, S1, S2 = ref
    u = torch.finfo(got_o.dtype).eps / 2
    go, gl = got_o.double().cpu().numpy(), got_lse.double().cpu().numpy()
    ds = 2.0 ** -15 * S1 + 2.0 ** -16 * S2
    seen = np.isfinite(lse)
    assert np.array_equal(np.isneginf(gl), np.isneginf(lse)), f"{what}: -inf pattern of lse"
    assert np.array_equal(np.isnan(gl), np.isnan(lse)), f"{what}: NaN pattern of lse"
    err = np.abs(gl - lse)[seen]
    tol = (ds + 2.0 ** -20 * (1 + np.abs(lse)))[seen]
    assert np.all(err <= tol), f"{what}: lse off by {(err / tol).max():.2f} of its bound"
    assert np.array_equal(np.isnan(go), np.isnan(o)), f"{what}: NaN pattern of o"
    fine = np.isfinite(o)
    dst = ds.T[:, :, None]
    tol = u * np.abs(o) + (1 + u) * (2.0 ** -11 + 2.0 ** -12 + 2 * dst) * A + 1e-30
    over = (np.abs(go - o) / tol)[fine]
    assert over.size == 0 or over.max() <= 1, f"{what}: o off by {over.max():.2f} of its bound"
    empty = np.isneginf(lse).T
    assert np.all(go[empty] == 0), f"{what}: rows that see nothing must be 0"
