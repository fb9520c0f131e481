"""Page calls refuse arrays that lie in the table or the lengths, which they write (on the host, no launch is made)."""
import pytest

from test_cache_abi import INVALID, WS, bd, calls, view  # noqa: F401  (bd is a fixture)

# view(bd): 3 sequences of 4 entries: table is [4096, 4144), lens [8192, 8204)


@pytest.mark.parametrize("name,kw", [
    ("reserve", dict(new=4096)), ("reserve", dict(new=4140)), ("reserve", dict(new=4088)),
    ("reserve", dict(new=8196)), ("reserve", dict(new=8184)), ("reserve", dict(new=8200)),
    ("fork", dict(p=4100)), ("fork", dict(p=8192)), ("fork", dict(k=4092)), ("fork", dict(k=8200)), ("fork", dict(lens=4096)),
    ("fork", dict(lens=4140)), ("compact", dict(live=4096)), ("compact", dict(live=8200))])
def test_arrays_in_what_the_call_writes(bd, name, kw):
    assert calls(bd)[name](view(bd), **kw) == INVALID
    assert bd.bdlm_last_launch_count() == 0


@pytest.mark.parametrize("name,kw", [
    ("reserve", dict(new=8192)), ("reserve", dict(new=8204)), ("reserve", dict(new=8180)), ("reserve", dict(new=4144)),
    ("reserve", dict(new=4084)), ("fork", dict(lens=8192)), ("fork", dict(p=8204, k=8184)), ("compact", dict(live=4144))])
def test_arrays_beside_it_pass_on_to_the_next_check(bd, name, kw):
    assert calls(bd)[name](view(bd), ws=None, **kw) == WS
    assert bd.bdlm_last_launch_count() == 0
