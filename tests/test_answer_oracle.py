"""Pins of the answering oracle: worked examples, and the cut into runs against every cut there is."""
import itertools
import math

import numpy as np
import pytest

from oracle import answer_oracle as ao

X = [math.log(w) for w in (1.0, 4.0, 2.0, 1.0)]  # by number; ranked: 1, 2, 0, 3


@pytest.mark.parametrize("u,kw,want", [
    (0.0, {}, 0), (0.124, {}, 0), (0.126, {}, 1), (0.62, {}, 1), (0.63, {}, 2), (0.874, {}, 2), (0.876, {}, 3), (1.0, {}, 3),
    (0.0, dict(top_k=2), 1), (0.66, dict(top_k=2), 1), (0.67, dict(top_k=2), 2), (0.0, dict(top_k=3), 0), (0.99, dict(top_k=3), 2),
    (0.9, dict(top_p=0.4), 1), (0.9, dict(top_p=0.6), 2), (0.99, dict(top_p=0.8), 2), (0.0, dict(top_p=0.8), 0), (0.5, dict(top_p=0.0), 1),
    (0.0, dict(min_p=0.3), 1), (0.99, dict(min_p=0.3), 2), (0.99, dict(min_p=2.0), 1), (0.5, dict(temperature=0.0), 1),
    (0.0, dict(top_k=3, top_p=0.5), 1), (0.99, dict(top_k=3, top_p=0.5), 1), (0.99, dict(top_k=3, top_p=0.6), 2)])
def test_sample(u, kw, want):
    token, lp = ao.sample_row(X, u, **kw)
    assert token == want and lp == pytest.approx(X[want] - math.log(8.0), abs=1e-14)


def test_sample_edges():
    nan, inf = math.nan, math.inf
    assert ao.sample_row([-inf, nan], 0.5) == (-1, -inf)
    assert ao.sample_row([0.0, inf, 5.0, inf], 0.6) == (3, pytest.approx(-math.log(2)))
    assert ao.sample_row([nan, 1.0, -inf], 0.9) == (1, 0.0)
    assert ao.sample_row([2.0, 2.0, 2.0], 0.9, top_k=2)[0] == 1
    assert ao.sample_row([0.0, -0.0], 0.9, top_k=1)[0] == 0


def test_unmask():
    now, got, lp = [9, 9, 5, 9, 9, 9], [1, 2, 3, 4, -1, 6], [-1.0, -0.5, 0.0, -0.5, 0.0, math.nan]
    for n_min, thr, want in ((0, -0.6, [9, 2, 5, 4, 9, 9]), (1, -0.1, [9, 2, 5, 9, 9, 9]), (3, -0.6, [1, 2, 5, 4, 9, 9]),
                             (9, 0.0, [1, 2, 5, 4, 9, 6]), (0, math.nan, now), (2, math.nan, [9, 2, 5, 4, 9, 9])):
        out, left = ao.unmask(now, got, lp, [0, 5, 6], 9, [n_min, 0], [thr, -9.0])
        if n_min == 9:
            want = want[:5] + [9]
        assert out.tolist() == want and left.tolist() == [want[:5].count(9), 1]


@pytest.mark.parametrize("seed", range(60))
def test_runs_save_most(seed):
    rng = np.random.default_rng(seed)
    m, longest = int(rng.integers(1, 9)), int(rng.integers(2, 10))
    c = rng.integers(0, 6, m - 1).tolist()
    n = m + int(rng.integers(0, 3))
    busy = sorted(rng.choice(n, m, replace=False).tolist())
    rows = [int(s in busy) for s in range(n)]
    plan = ao.runs(busy, c, n, 16, longest)
    most = 0
    for cuts in itertools.product([0, 1], repeat=m - 1):
        edges = [0] + [i + 1 for i, x in enumerate(cuts) if x] + [m]
        if max(b - a for a, b in zip(edges, edges[1:])) <= longest:
            most = max(most, sum((b - a - 1) * min(c[a:b - 1], default=0) for a, b in zip(edges, edges[1:])))
    assert ao.saved(plan, rows, 16) == most
    for s in range(n):  # every sequence of a run names the same one
        first, end, shared = plan[:, s]
        assert first <= s < end and np.all(plan[:, first:end] == plan[:, s:s + 1])
        if shared:
            inside = [i for i in range(m) if first <= busy[i] < end]
            assert len(inside) > 1 and shared == 16 * min(c[i] for i in inside[:-1])


def test_unmask_keeps_no_mask():
    out, left = ao.unmask([9, 9, 9, 4], [9, 1, 2, 3], [0.0, -1.0, -2.0, 0.0], [0, 4], 9, [1], [-0.5])
    assert out.tolist() == [9, 1, 9, 4] and left.tolist() == [2]
