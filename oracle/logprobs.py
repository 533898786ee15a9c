"""Binary64 oracle of token log probabilities, their gradient and cache eviction.

TEST INFRASTRUCTURE ONLY, like the rest of this package: plain row-at-a-time arithmetic from the formulas, sharing
nothing with the HIP library. [LOGP] ("Design: the numeric contract", "Contract constants") fixes the log-sum-exp over
the whole row with -inf contributing 0 and the temperature in the exponent; [DETK] ("Changes") the order: value
descending, then index ascending.
"""
from __future__ import annotations

import math
from dataclasses import dataclass
from typing import List, Optional

import numpy as np

STATUS_OK = 0
STATUS_NONFINITE = 1
STATUS_BAD_K = 2
STATUS_BAD_T = 4
STATUS_BAD_TOKEN = 6


@dataclass
class LogpResult:
    status: int
    logp: float = math.nan
    rank: int = -1
    entropy: float = math.nan
    lse: float = math.nan
    top_idx: Optional[List[int]] = None
    top_logp: Optional[List[float]] = None


def _exponents(x: np.ndarray, t: float) -> np.ndarray:
    with np.errstate(over="ignore"):
        return (x - x.max()) / t


def token_logp_row(row, t: float = 1.0, token: int = -1, n_top: int = 0) -> LogpResult:
    """One row: status, logp and rank of `token` (-1: none), entropy, lse and the best n_top tokens."""
    x = np.asarray(row, dtype=np.float64)
    poisoned = dict(top_idx=[-1] * n_top, top_logp=[math.nan] * n_top)
    if np.isnan(x).any() or (x == math.inf).any() or (x == -math.inf).all():
        return LogpResult(STATUS_NONFINITE, **poisoned)
    if not 0.0 <= t < math.inf:
        return LogpResult(STATUS_BAD_T, **poisoned)
    if token != -1 and not 0 <= token < len(x):
        return LogpResult(STATUS_BAD_TOKEN, **poisoned)
    order = np.lexsort((np.arange(len(x)), -x))                    # value descending, id ascending
    rank = 0 if token < 0 else int(np.nonzero(order == token)[0][0]) + 1
    best = [int(i) for i in order[:n_top] if x[i] > -math.inf]
    pad = n_top - len(best)
    if t == 0.0:
        logp = 0.0 if rank in (0, 1) else -math.inf
        top = [0.0 if i == 0 else -math.inf for i in range(len(best))]
        return LogpResult(STATUS_OK, logp, rank, 0.0, math.inf, best + [-1] * pad, top + [-math.inf] * pad)
    d = _exponents(x, t)
    e = np.exp(d)
    s = math.fsum(e)
    live = e > 0
    entropy = math.log(s) - math.fsum(e[live] * d[live]) / s
    logp = 0.0 if token < 0 else min(d[token] - math.log(s), 0.0)
    top = [min(d[i] - math.log(s), 0.0) for i in best]
    return LogpResult(STATUS_OK, float(logp), rank, max(entropy, 0.0), float(x.max() / t + math.log(s)), best + [-1] * pad,
                      [float(v) for v in top] + [-math.inf] * pad)


def token_logp_grad_row(row, t: float, token: int, a: float, h: float, l: float) -> np.ndarray:
    """Gradient of a * logp + h * entropy + l * lse with respect to one (valid) row; a is ignored without a token."""
    x = np.asarray(row, dtype=np.float64)
    if t == 0.0:
        return np.zeros_like(x)
    d = _exponents(x, t)
    p = np.exp(d)
    p /= math.fsum(p)
    live = p > 0
    mean = math.fsum(p[live] * d[live])
    a = a if token >= 0 else 0.0
    g = np.where(live, p * (l - a - h * (np.where(live, d, 0.0) - mean)), 0.0)
    if token >= 0:
        g[token] += a
    return g / t


@dataclass
class EvictResult:
    status: int
    source: List[int]
    score: Optional[np.ndarray] = None
    position: Optional[np.ndarray] = None
    length: int = 0


def cache_evict_row(score, weights, position, n: int, keep: int, keep_max: int, sinks: int, recent: int) -> EvictResult:
    """One cache row. score [slots], weights [n_w, slots], position [slots]; n: slots in use. The results are the new
    length and, for each slot below it, the slot its contents come from, its fp32 weight and its position."""
    total = []
    for j in range(n):
        s = float(score[j])
        for w in range(len(weights)):
            s += float(weights[w][j])
        total.append(float(np.float32(s)))
    if any(not math.isfinite(s) for s in total):
        return EvictResult(STATUS_NONFINITE, [], length=n)
    k = min(keep, n)
    if keep < 1 or k > keep_max:
        return EvictResult(STATUS_BAD_K, [], length=n)
    newest = max((int(position[j]) for j in range(n)), default=0)
    protected = [int(position[j]) < sinks or int(position[j]) > newest - recent for j in range(n)]
    kept = set(sorted(range(n), key=lambda j: (not protected[j], -total[j], j))[:k])
    fillers = iter(j for j in range(k, n) if j in kept)
    source = [j if j in kept else next(fillers) for j in range(k)]
    return EvictResult(STATUS_OK, source, np.array([total[j] for j in source], np.float32),
                       np.array([position[j] for j in source], np.int32), k)


def cache_evict_row_sorted(score, weights, position, n: int, keep: int, keep_max: int, sinks: int, recent: int) -> EvictResult:
    """cache_evict_row for long rows: the same by one numpy sort of all slots (pinned against it)."""
    total = np.array(score[:n], np.float64)
    for w in weights:
        total += np.asarray(w[:n], np.float64)
    with np.errstate(over="ignore"):
        total = total.astype(np.float32)
    if not np.isfinite(total).all():
        return EvictResult(STATUS_NONFINITE, [], length=n)
    k = min(keep, n)
    if keep < 1 or k > keep_max:
        return EvictResult(STATUS_BAD_K, [], length=n)
    place = np.asarray(position[:n], np.int64)
    protected = (place < sinks) | (place > place.max(initial=0) - recent)
    order = np.lexsort((np.arange(n), -total, ~protected))
    stays = np.zeros(n, bool)
    stays[order[:k]] = True
    source = np.arange(k)
    source[~stays[:k]] = k + np.nonzero(stays[k:])[0]
    return EvictResult(STATUS_OK, source.tolist(), total[source], place[source].astype(np.int32), k)
