"""That the caches of cache_marks are what they say, and that their bounds do see a lost and a repeated tile, whichever it
is (on the CPU, the mistake made in the expected results)."""
import numpy as np
import pytest
import torch

from oracle import cache_oracle as co

import cache_marks as cm
import cache_util as cu


@pytest.mark.parametrize("keys", ["any", "alike"])
@pytest.mark.parametrize("name", list(cm.CASES))
def test_a_lost_or_repeated_tile_breaks_the_bounds(name, keys):
    lens, rows, _, _, _, d, block = cm.CASES[name]
    c, off, q, qh = cm.make(name, keys)
    ref = co.attention(c, 0, qh, off, block, d ** -0.5)
    o, lse = cm.closed_form(name, c, qh)
    for dtype in (torch.bfloat16, torch.float32):
        as_out = lambda o: torch.from_numpy(o).to(dtype)
        cu.check_attention(as_out(o), torch.from_numpy(lse).float(), ref)
    for s in range(0, len(lens), max(1, len(lens) // 8)):
        n = lens[s]
        seen = min(n, ((n - 1) // block + 1) * block)
        for t in range(-(-seen // cm.TILE)):
            for how in ("lose", "repeat"):
                bad_o, bad_lse = cm.closed_form(name, c, qh, **{how: (s, t)})
                rows_of_s = slice(off[s], off[s + 1])
                part = [x[rows_of_s] if i in (0, 2) else x[:, rows_of_s] for i, x in enumerate(ref)]
                with pytest.raises(AssertionError):
                    cu.check_attention(torch.from_numpy(bad_o[rows_of_s]).bfloat16(),
                                       torch.from_numpy(bad_lse[:, rows_of_s]).float(), part)
