"""What a call with runs asks for beyond one without (no GPU needed)."""
import pytest

from test_cache_abi import bd  # noqa: F401  (a fixture)


@pytest.mark.parametrize("rows,heads,kv_heads,d,n", [(69500, 32, 8, 128, 16), (1 << 20, 64, 8, 64, 64), (4096, 4, 4, 128, 1), (3, 8, 1, 64, 900),
                                                     (32, 32, 8, 128, 8), (33, 32, 8, 128, 1), (1 << 26, 16, 1, 64, 65536)])
def test_planes_hold_what_can_be_read_together(bd, rows, heads, kv_heads, d, n):
    """Two planes of at most 128 flat rows for each sequence and kv head, or of all rows where those are fewer."""
    alone = bd.bdlm_cache_attn_fwd_workspace_bytes(rows, heads, kv_heads, d, n)
    flat = min(rows * heads // kv_heads, 128 * n)
    more = bd.bdlm_cache_attn_shared_fwd_workspace_bytes(rows, heads, kv_heads, d, n) - alone
    assert alone > 0 and 2 * 4 * kv_heads * flat * (d + 1) <= more < 2 * 4 * kv_heads * flat * (d + 1) + 256
