"""Pins of the binary64 oracles of token log probabilities, their gradient and cache eviction (no GPU)."""
import itertools
import math

import numpy as np
import pytest
from scipy import special, stats

import oracle


@pytest.mark.parametrize("v,t", [(1, 1.0), (2, 0.3), (17, 1.0), (1000, 1.7)])
def test_logp_against_scipy(v, t):
    rng = np.random.default_rng(v)
    x = rng.standard_normal(v) * 3
    if v > 2:
        x[rng.integers(0, v, v // 4)] = -np.inf
        x[0] = 0.5
    for token in range(min(v, 5)):
        r = oracle.token_logp_row(x, t, token, 3)
        lse = special.logsumexp(x / t)
        assert r.status == 0 and r.lse == pytest.approx(lse, abs=1e-12)
        assert r.logp == pytest.approx(x[token] / t - lse, abs=1e-12)
        assert r.entropy == pytest.approx(stats.entropy(special.softmax(x / t)), abs=1e-12)
        assert r.rank == 1 + int((x > x[token]).sum() + (x[:token] == x[token]).sum())
    assert r.top_idx[0] == int(np.argmax(x)) and r.top_logp[0] == pytest.approx(x.max() / t - lse, abs=1e-12)


def test_logp_closed_forms():
    r = oracle.token_logp_row(np.zeros(8), 2.0, 5, 3)
    assert r.logp == pytest.approx(-math.log(8)) and r.entropy == pytest.approx(math.log(8)) and r.rank == 6
    assert r.top_idx == [0, 1, 2]                                  # equal values: lowest ids first
    r = oracle.token_logp_row([1.0, -math.inf, 4.0], 0.0, 2, 3)     # greedy
    assert (r.logp, r.rank, r.entropy, r.lse) == (0.0, 1, 0.0, math.inf)
    assert r.top_idx == [2, 0, -1] and r.top_logp == [0.0, -math.inf, -math.inf]
    assert oracle.token_logp_row([1.0, 4.0], 0.0, 0).logp == -math.inf
    r = oracle.token_logp_row([0.0, -math.inf], 1.0, 1, 2)
    assert r.logp == -math.inf and r.rank == 2 and r.entropy == 0.0 and r.top_idx == [0, -1]
    for bad in ([math.nan, 1.0], [math.inf, 1.0], [-math.inf, -math.inf]):
        assert oracle.token_logp_row(bad, 1.0, 0).status == oracle.STATUS_NONFINITE
    assert oracle.token_logp_row([1.0], -1.0, 0).status == oracle.STATUS_BAD_T
    assert oracle.token_logp_row([1.0], 1.0, 1).status == oracle.STATUS_BAD_TOKEN
    assert oracle.token_logp_row([1.0], 1.0, -2).status == oracle.STATUS_BAD_TOKEN
    assert oracle.token_logp_row([1.0, 2.0], 1.0, -1).rank == 0


@pytest.mark.parametrize("t", [0.5, 1.0, 3.0])
def test_gradient_against_central_differences(t):
    rng = np.random.default_rng(3)
    x = rng.standard_normal(9)
    x[4] = -np.inf
    for token, a, h, l in [(2, 1.0, 0.0, 0.0), (-1, 5.0, 1.0, 0.0), (0, 0.0, 0.0, 1.0), (7, -0.7, 0.3, 0.2)]:
        def loss(y):
            r = oracle.token_logp_row(y, t, token)
            return (a * r.logp if token >= 0 else 0.0) + h * r.entropy + l * r.lse
        g = oracle.token_logp_grad_row(x, t, token, a, h, l)
        assert g[4] == 0.0
        step = 1e-5
        for i in range(9):
            if i == 4:
                continue
            up, dn = x.copy(), x.copy()
            up[i] += step
            dn[i] -= step
            # a central difference is off by step^2 / 6 times the third derivative and by rounding over 2 step
            assert g[i] == pytest.approx((loss(up) - loss(dn)) / (2 * step), abs=2e-9), (token, i)
    assert not oracle.token_logp_grad_row(x, 0.0, 2, 1.0, 1.0, 1.0).any()


def test_evict_against_enumeration():
    # the kept set is the one whose sorted (protected, weight, -slot) tuples are the largest of all sets of its size
    rng = np.random.default_rng(5)
    for trial in range(60):
        n, keep = int(rng.integers(1, 8)), int(rng.integers(1, 9))
        score = rng.integers(0, 3, 8).astype(np.float32)
        w = rng.integers(0, 2, (2, 8)).astype(np.float32)
        position = rng.permutation(8).astype(np.int32)
        sinks, recent = int(rng.integers(0, 3)), int(rng.integers(0, 4))
        r = oracle.cache_evict_row(score, w, position, n, keep, 8, sinks, recent)
        total = (score + w.sum(0))[:n]
        newest = position[:n].max()
        worth = [(position[j] < sinks or position[j] > newest - recent, total[j], -j) for j in range(n)]
        k = min(keep, n)
        best = max(itertools.combinations(range(n), k), key=lambda c: sorted((worth[j] for j in c), reverse=True))
        assert r.status == 0 and r.length == k and sorted(r.source) == list(best)
        assert all(r.source[j] == j for j in range(k) if j in best)       # kept slots stay in place
        moved = [r.source[j] for j in range(k) if j not in best]
        assert moved == sorted(moved) and all(j >= k for j in moved)
        assert np.array_equal(r.score, total[r.source]) and np.array_equal(r.position, position[r.source])


def test_evict_edges():
    r = oracle.cache_evict_row([1.0], [], [0], 0, 3, 3, 1, 1)
    assert (r.status, r.source, r.length) == (0, [], 0)
    assert oracle.cache_evict_row([math.nan, 1.0], [], [0, 1], 2, 1, 1, 0, 0).status == oracle.STATUS_NONFINITE
    assert oracle.cache_evict_row([1.0, math.nan], [], [0, 1], 1, 1, 1, 0, 0).status == 0     # behind the length
    assert oracle.cache_evict_row([1.0, 2.0], [], [0, 1], 2, 0, 1, 0, 0).status == oracle.STATUS_BAD_K
    assert oracle.cache_evict_row([1.0, 2.0], [], [0, 1], 2, 2, 1, 0, 0).status == oracle.STATUS_BAD_K


def test_evict_by_one_sort_equals_the_plain_oracle():
    rng = np.random.default_rng(6)
    for trial in range(120):
        slots, keep = int(rng.integers(1, 40)), int(rng.integers(0, 42))
        n, keep_max = int(rng.integers(0, slots + 1)), int(rng.integers(1, 42))
        score = rng.integers(-1, 3, slots).astype(np.float32) if trial % 2 else rng.standard_normal(slots).astype(np.float32)
        if trial % 7 == 0:
            score[rng.integers(0, slots)] = [math.nan, math.inf, -math.inf, 3e38][trial % 4]
        w = rng.random((trial % 3, slots)).astype(np.float32) * (3e38 if trial % 11 == 0 else 1)
        position = rng.permutation(slots).astype(np.int32) - (20 if trial % 5 == 0 else 0)
        args = (score, w, position, n, keep, keep_max, int(rng.integers(0, 9)), int(rng.choice([0, 3, 30, 2 ** 31 - 1])))
        a, b = oracle.cache_evict_row(*args), oracle.cache_evict_row_sorted(*args)
        assert (a.status, a.source, a.length) == (b.status, b.source, b.length), trial
        if not a.status:
            assert np.array_equal(a.score, b.score) and np.array_equal(a.position, b.position), trial
