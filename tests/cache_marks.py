"""Caches over which a lost or repeated tile of keys shows: every key that a row sees weighs the same (queries of zeros, or
keys that are all alike), so that the score errors of the bounds in cache_util are next to nothing, and the values of
tile t of 128 keys have one entry that is not 0, 2^((t / d) % 4) in column t % d."""
import numpy as np
import torch

from oracle import cache_oracle as co

import cache_util as cu

TILE = 128
# lens, rows, page, G, Hk, d, block; flat rows of a unit are rows * G
CASES = {
    "one row, 235 tiles": ([30011], [1], 64, 4, 1, 128, 32),
    "nine rows, 235 tiles": ([30011], [9], 64, 4, 1, 128, 32),
    "two-tile unit, 235 tiles": ([30011], [64], 64, 4, 1, 128, 32),
    "five rows, causal": ([20000], [5], 32, 3, 1, 128, 1),
    "two-tile unit, half alive": ([12929], [40], 16, 4, 2, 64, 8),
    "multiples of a tile": ([127, 128, 129, 255, 256, 257, 383, 384, 385, 4095, 4096, 4097], [1] * 12, 16, 2, 2, 64, 1),
    "multiples of a tile, two-tile units": ([383, 384, 385, 2047, 2048, 2049], [70] * 6, 128, 2, 1, 128, 16),
    "24 sequences": ([1400 + 37 * s for s in range(24)], [2] * 24, 64, 8, 1, 128, 32),
    "24 sequences, two-tile units": ([1400 + 37 * s for s in range(24)], [32] * 24, 64, 8, 1, 128, 32),
    "a prompt of several units": ([1500], [900], 128, 1, 2, 128, 48),
}


def make(name, keys):
    """keys: "alike" or "any" (queries of zeros). Returns (cache, offsets, q bf16 on the host, q float64)."""
    lens, rows, page, G, Hk, d, block = CASES[name]
    c = cu.make(len(name), lens=lens, page=page, Hk=Hk, d=d)
    rng = np.random.default_rng(7)
    q = rng.standard_normal((sum(rows), G * Hk, d)) * (0.3 if keys == "alike" else 0.0)
    if keys == "alike":
        c["k"][:] = rng.integers(0x28, 0x40, (1, 1, Hk, 1, d), dtype=np.uint8)  # 2^-2 .. 1.875
        c["ks"][:] = 1.0
    c["v"][:], c["vs"][:] = 0, 1.0
    for s, n in enumerate(lens):
        for j in range(n):
            t = j // TILE
            c["v"][0, c["table"][s, j // page], :, j % page, t % d] = 0x38 + 8 * (t // d % 4)
    q = torch.from_numpy(q).bfloat16()
    return c, cu.offsets(rows), q, q.double().numpy()


def closed_form(name, c, qh, lose=None, repeat=None):
    """(o, lse) of the case, with tile `lose` or `repeat` = (sequence, tile) counted not at all or twice."""
    lens, rows, page, G, Hk, d, block = CASES[name]
    T, H, _ = qh.shape
    o, lse = np.zeros((T, H, d)), np.zeros((H, T))
    tiles = np.arange(-(-max(lens) // TILE))
    marks = np.zeros((len(tiles), d))
    marks[tiles, tiles % d] = 2.0 ** (tiles // d % 4)
    k0 = co.VALUES[c["k"][0, c["table"][0, 0], :, 0]] * c["ks"][0, c["table"][0, 0], :, None]
    at = 0
    for s, (n, r) in enumerate(zip(lens, rows)):
        for i in range(r):
            end = min(n, ((n - r + i) // block + 1) * block)
            keys = np.clip(end - TILE * tiles, 0, TILE).astype(np.float64)
            for what, f in ((lose, 0), (repeat, 2)):
                if what is not None and what[0] == s:
                    keys[what[1]] *= f
            with np.errstate(invalid="ignore", divide="ignore"):  # the only tile is lost
                o[at] = keys @ marks / keys.sum()
                lse[:, at] = (qh[at] * np.repeat(k0, G, 0)).sum(1) * d ** -0.5 + np.log(keys.sum())
            at += 1
    return o, lse
