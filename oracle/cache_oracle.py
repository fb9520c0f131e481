"""Float64 oracle of the paged 8-bit cache: e4m3 codes from their definition,
writing rows with power-of-two scales, block-causal attention over the cache,
and the page calls. Plain loops over numpy arrays, none of the library's code.

A cache is a dict of numpy arrays: k, v uint8 codes [layers, pages, Hk, page, d];
ks, vs float64 scales [layers, pages, Hk]; table int [seqs, max_pages]; lens.
"""
import math

import numpy as np


def e4m3_value(code: int) -> float:
    """1 sign, 4 exponent (bias 7), 3 mantissa bits; 0x7f and 0xff are NaN."""
    e, m = (code >> 3) & 15, code & 7
    if e == 15 and m == 7:
        return math.nan
    x = math.ldexp(m, -9) if e == 0 else math.ldexp(8 + m, e - 10)
    return -x if code & 128 else x


VALUES = np.array([e4m3_value(c) for c in range(256)])


def encode(x):
    """Codes nearest to x (|x| <= 448), ties to the even code; NaN (0x7f) for
    what is not finite."""
    x = np.asarray(x, dtype=np.float64)
    a = np.where(np.isfinite(x), np.abs(x), 0.0)
    up = VALUES[:127]
    hi = np.minimum(np.searchsorted(up, a), 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - up[lo], up[hi] - a
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi) | np.where(np.signbit(x), 128, 0)
    return np.where(np.isfinite(x), code, 127).astype(np.uint8)


def pow2_scale(amax: float) -> float:
    """The smallest power of two s >= 2^-126 with amax <= 448 s; 1 for 0."""
    if amax == 0:
        return 1.0
    s = 2.0 ** -126
    while amax > 448 * s:
        s *= 2
    return s


def pages_of(n: int, page: int) -> int:
    return -(-int(n) // page)


def write(c, layer, k_new, v_new, cu):
    """In place; k_new, v_new float64 [T, Hk, d]."""
    page = c["k"].shape[3]
    for s in range(len(c["lens"])):
        r, n = int(cu[s + 1] - cu[s]), int(c["lens"][s])
        if r == 0:
            continue
        for j in range((n - r) // page, pages_of(n, page)):
            pid = int(c["table"][s, j])
            for codes, scales, new in ((c["k"], c["ks"], k_new), (c["v"], c["vs"], v_new)):
                for h in range(codes.shape[2]):
                    x = VALUES[codes[layer, pid, h]] * scales[layer, pid, h]
                    rows = min(page, n - j * page)
                    for i in range(rows):
                        pos = j * page + i
                        if pos >= n - r:
                            x[i] = new[cu[s] + pos - (n - r), h]
                    x = x[:rows]
                    fin = np.abs(x[np.isfinite(x)])
                    sc = pow2_scale(float(fin.max()) if fin.size else 0.0)
                    old = scales[layer, pid, h]
                    kept = max(0, min(rows, n - r - j * page))
                    if sc != old:
                        codes[layer, pid, h, :kept] = encode(x[:kept] / sc)
                    codes[layer, pid, h, kept:rows] = encode(x[kept:] / sc)
                    scales[layer, pid, h] = sc


def attention(c, layer, q, cu, block, scale, q_pos=None):
    """(o, lse, A, S1, S2) of the rows q [T, H, d]; for error bounds A = sum_j
    p_j |v_j| per entry of o, S1 = max_j scale sum_c |q_c k_jc| and S2 = scale
    d max_c |q_c| max_jc |k_jc| per row, over the keys that the row sees."""
    q = np.asarray(q, dtype=np.float64)
    T, H, d = q.shape
    Hk, page = c["k"].shape[2], c["k"].shape[3]
    o, A = np.zeros((T, H, d)), np.zeros((T, H, d))
    lse, S1, S2 = np.full((H, T), -np.inf), np.zeros((H, T)), np.zeros((H, T))
    for s in range(len(c["lens"])):
        n, a, b = int(c["lens"][s]), int(cu[s]), int(cu[s + 1])
        if b == a:
            continue
        ids = c["table"][s, :pages_of(n, page)]
        start = n - (b - a) if q_pos is None else int(q_pos[s])
        for h in range(Hk):
            k = (VALUES[c["k"][layer, ids, h]] * c["ks"][layer, ids, h][:, None, None]).reshape(-1, d)[:n]
            v = (VALUES[c["v"][layer, ids, h]] * c["vs"][layer, ids, h][:, None, None]).reshape(-1, d)[:n]
            for i in range(a, b):
                end = min(n, ((start + i - a) // block + 1) * block)
                if end == 0:
                    continue
                kk, vv = k[:end], v[:end]
                for g in range(h * (H // Hk), (h + 1) * (H // Hk)):
                    with np.errstate(invalid="ignore"):
                        x = scale * (kk @ q[i, g])
                        m = x.max()
                        p = np.exp(x - m)
                        z = p.sum()
                        o[i, g] = (p @ vv) / z
                        A[i, g] = (p @ np.abs(vv)) / z
                        lse[g, i] = m + np.log(z)
                        S1[g, i] = scale * (np.abs(kk) @ np.abs(q[i, g])).max()
                        S2[g, i] = scale * d * np.abs(q[i, g]).max() * np.abs(kk).max()
    return o, lse, A, S1, S2


def live_pages(c, lens=None):
    """Users of every page: sequences whose first ceil(len / page) entries name it."""
    page, users = c["k"].shape[3], np.zeros(c["k"].shape[1], dtype=int)
    for s, n in enumerate(c["lens"] if lens is None else lens):
        for i in c["table"][s, :pages_of(n, page)]:
            users[i] += 1
    return users


def reserve(c, new_lens):
    """In place; returns "" or why nothing was changed."""
    page, cap = c["k"].shape[3], c["table"].shape[1]
    if any(n < 0 or pages_of(n, page) > cap for n in new_lens):
        return "length"
    users = live_pages(c, np.minimum(c["lens"], new_lens))
    free = [i for i, u in enumerate(users) if u == 0]
    need = [max(0, pages_of(b, page) - pages_of(a, page)) for a, b in zip(c["lens"], new_lens)]
    for s, (a, b) in enumerate(zip(c["lens"], new_lens)):
        if b > a and a % page and users[c["table"][s, a // page]] > 1:
            return "shared"
    if sum(need) > len(free):
        return "pages"
    for s, n in enumerate(need):
        at = pages_of(c["lens"][s], page)
        c["table"][s, at:at + n], free = free[:n], free[n:]
        c["lens"][s] = new_lens[s]
    return ""


def fork(c, parents, children, fork_lens=None):
    page = c["k"].shape[3]
    n = [int(c["lens"][p]) for p in parents] if fork_lens is None else [int(x) for x in fork_lens]
    if len(set(children)) != len(children) or set(children) & set(parents):
        return "children"
    if any(c["lens"][k] for k in children) or any(x < 0 or x > c["lens"][p] for x, p in zip(n, parents)):
        return "length"
    free = [i for i, u in enumerate(live_pages(c)) if u == 0]
    if sum(x % page > 0 for x in n) > len(free):
        return "pages"
    for x, p, k in zip(n, parents, children):
        full, tail = x // page, x % page
        c["table"][k, :full] = c["table"][p, :full]
        if tail:
            src, dst = int(c["table"][p, full]), free.pop(0)
            c["table"][k, full] = dst
            for name in "kv":
                c[name][:, dst, :, :tail] = c[name][:, src, :, :tail]
                c[name + "s"][:, dst] = c[name + "s"][:, src]
        c["lens"][k] = x
    return ""


def compact(c):
    """In place; returns the number of live pages."""
    page, users = c["k"].shape[3], live_pages(c)
    live = int((users > 0).sum())
    holes = [i for i in range(live) if users[i] == 0]
    movers = [i for i in range(live, len(users)) if users[i] > 0]
    to = dict(zip(movers, holes))
    for src, dst in to.items():
        for name in ("k", "v", "ks", "vs"):
            c[name][:, dst] = c[name][:, src]
    for s, n in enumerate(c["lens"]):
        for i in range(pages_of(n, page)):
            c["table"][s, i] = to.get(int(c["table"][s, i]), c["table"][s, i])
    return live
