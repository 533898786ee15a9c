"""GPU tests of ts_cache_evict on rows up to the longest it takes, 2^22 slots, and of cuts through a crowd of nearly or
exactly equal weights, against the oracle: what stays, where it goes and its weights, equal in every bit."""
import numpy as np
import pytest

import oracle
import top_select_gumbel_amd as ts
from gpu_helpers import banner, host, torch_cuda

pytestmark = pytest.mark.gpu
LISTED = 4096        # slots of the cut's first bin that are listed; more take another path
RANKED = 256         # slots of a later bin that are ranked; more are binned again
BITS = 11            # a bin's


def check(score, keep, weights=None, wtype="float16", lengths=None, keeps=None, sinks=0, recent=0, dim=3, seed=0, in_place=False):
    torch = torch_cuda()
    rows, slots = score.shape
    banner(f"evict long rows={rows} slots={slots} keep={keep} sinks={sinks} recent={recent}")
    rng = np.random.default_rng(seed)
    position = np.stack([rng.permutation(slots) for _ in range(rows)]).astype(np.int32)
    lengths = np.full(rows, slots, np.int32) if lengths is None else np.asarray(lengths, np.int32)
    keeps = np.full(rows, keep, np.int32) if keeps is None else np.asarray(keeps, np.int32)
    w = None if weights is None else torch.from_numpy(weights).to(getattr(torch, wtype)).cuda()
    cache = torch.from_numpy(rng.integers(0, 256, (1, rows, slots, dim), dtype=np.uint8)).cuda()
    was = host(cache)
    r = ts.ts_cache_evict(*(torch.from_numpy(a.copy()).cuda() for a in (score, position, lengths, keeps)), keep, weights=w, k_cache=cache,
                          sinks=sinks, recent=recent, in_place=in_place)
    torch.cuda.synchronize()
    src, length, sc, pos, st = (host(t) for t in r)
    now, ws = host(cache), np.zeros((rows, 0, slots)) if w is None else w.double().cpu().numpy()
    for i in range(rows):
        o = oracle.cache_evict_row_sorted(score[i], ws[i], position[i], int(lengths[i]), int(keeps[i]), keep, sinks, recent)
        assert st[i] == o.status == 0 and length[i] == o.length, i
        m = o.length
        assert np.array_equal(src[i, :m], o.source) and (src[i, m:] == -1).all(), i
        assert np.array_equal(sc[i, :m].view(np.uint32), o.score.view(np.uint32)) and not sc[i, m:keep].any(), i
        assert np.array_equal(pos[i, :m], o.position) and (pos[i, m:keep] == -1).all(), i
        assert np.array_equal(now[0, i, :m], was[0, i][np.array(o.source)]) and np.array_equal(now[0, i, m:], was[0, i, m:]), i
        if in_place:
            assert np.array_equal(sc[i, keep:], score[i, keep:]) and np.array_equal(pos[i, keep:], position[i, keep:]), i


def weights_of(rng, rows, n, slots):
    """Accumulated weights over several octaves, a fifth of them exactly 0, and attention weights many of which underflow fp16."""
    score = np.exp(rng.standard_normal((rows, slots)) * 2 - 4).astype(np.float32)
    score[rng.random((rows, slots)) < 0.2] = 0
    w = np.exp(rng.standard_normal((rows, n, slots)) * 2.5)
    return score, (w / w.sum(-1, keepdims=True)).astype(np.float32)


@pytest.mark.parametrize("slots,rows", [(262144, 2), (262145, 2), (300000, 3), (1048577, 1), (1100000, 1), (1 << 22, 1)])
@pytest.mark.parametrize("share", [0.03, 0.45, 0.9])
def test_longest_rows(slots, rows, share):
    rng = np.random.default_rng(slots)
    score, w = weights_of(rng, rows, 1, slots)
    lengths = [slots - 777 * i for i in range(rows)]
    check(score, int(slots * share), w, lengths=lengths, sinks=4, recent=100, seed=slots)


def test_longest_row_of_which_one_goes_and_in_place():
    slots = 1 << 22
    rng = np.random.default_rng(1)
    score, _ = weights_of(rng, 1, 0, slots)
    check(score, slots - 1, seed=2, dim=1)
    check(score, slots // 2, seed=3, dim=1, in_place=True, lengths=[slots - 1])
    check(score, 1, seed=4, dim=1)


def crowd(rng, slots, equal, outlier):
    """Weights of which half or more share the row's bin of the cut, `equal` of them one value, and the number above that value."""
    s = (1 + rng.random(slots) / 32).astype(np.float32)
    at = rng.permutation(slots)
    one = np.float32(1 + 1 / 64)
    s[at[:equal]] = one
    s[at[-1]], s[at[-2]] = outlier, -outlier
    u = s.view(np.uint32).astype(np.int64)
    u = np.where(u >> 31, 0xFFFFFFFF ^ u, u | 0x80000000)
    u -= u.min()
    lo = int(u.max()).bit_length() - BITS
    mine = (u >> lo) == (u[at[0]] >> lo)
    return s, int((s > one).sum()), int((s == one).sum()), int(mine.sum()), lo


@pytest.mark.parametrize("slots", [20000, 70000, 300000])
@pytest.mark.parametrize("equal", [1, 200, 3000])
def test_cut_through_a_crowd(slots, equal):
    # an outlier stretches the bins, so that the cut's holds more than are listed; among them, further on, more equal ones than
    # are ranked, some of which stay
    rng = np.random.default_rng(slots + equal)
    s, above, same, in_bin, lo = crowd(rng, slots, equal, 1e30)
    assert in_bin > LISTED and lo > BITS and (equal < RANKED or same > RANKED)
    for keep in sorted({above + 1, above + (same + 1) // 2, above + same, above + same + 1, slots - 3}):
        check(s[None], keep, seed=keep)
        check(s[None], keep, seed=keep, sinks=2 ** 31 - 1)           # the cut among protected ones
        check(s[None], keep, seed=keep, sinks=50, recent=60, lengths=[slots - 1], in_place=True)


@pytest.mark.parametrize("slots", [20000, 131072, 1100000])
def test_cut_through_equal_weights(slots):
    # most of the cut's bin is one weight, 0: the lowest slots of them stay
    rng = np.random.default_rng(slots)
    score = np.exp(rng.standard_normal((2, slots)) * 2 - 4).astype(np.float32)
    score[rng.random((2, slots)) < 0.3] = 0
    for share in (0.75, 0.9, 0.99):
        check(score, int(slots * share), seed=1, dim=1)
    check(score, slots // 2, seed=2, dim=1, sinks=slots)
    # values next to each other: the last digit alone tells them apart
    near = (np.uint32(0x3F800000) + rng.integers(0, 3, (1, slots)).astype(np.uint32)).view(np.float32)
    near[0, 5] = 1e30
    for share in (0.2, 0.5, 0.8):
        check(near, int(slots * share), seed=3, dim=1)


def test_crowded_rows_beside_others():
    # rows that end each in its own way in one launch
    slots = 30000
    rng = np.random.default_rng(9)
    s, above, same, *_ = crowd(rng, slots, 3000, 1e30)
    rows = np.stack([s, np.full(slots, 2.5, np.float32), rng.random(slots).astype(np.float32), np.zeros(slots, np.float32), s])
    keep = above + same // 2
    check(rows, slots, keeps=[keep, 100, 7000, slots - 1, slots], lengths=[slots, slots, 29999, slots, 12345], dim=2, seed=5)
