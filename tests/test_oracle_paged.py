"""Pins of the paged cache's oracle: attention against torch's softmax in binary64 over the dense cache and closed forms; the
pages against the invariants that define them (every count is the number of entries that name the page, contents follow)."""
import numpy as np
import pytest

from oracle import paged


def cache(rng, pages, heads, slots, dim):
    return rng.standard_normal((pages, heads, slots, dim)), rng.standard_normal((pages, heads, slots, dim))


@pytest.mark.parametrize("hq,hk,n,window", [(4, 2, 11, 0), (3, 3, 7, 4), (6, 1, 12, 1)])
def test_attend_against_dense_softmax(hq, hk, n, window):
    torch = pytest.importorskip("torch")
    rng = np.random.default_rng(n)
    k, v = cache(rng, 9, hk, 4, 5)
    q = rng.standard_normal((hq, 5))
    table = rng.permutation(9)[:3]
    r = paged.attend_row(q, k, v, table, n, 0.3, window, 12)
    for h in range(hq):
        dense = [(x[table, h // (hq // hk)].reshape(12, 5))[max(0, n - window) if window else 0:n] for x in (k, v)]
        s = torch.from_numpy(dense[0] @ q[h] * 0.3)
        w = torch.softmax(s, 0).numpy()
        assert np.allclose(r.out[h], w @ dense[1], rtol=0, atol=1e-13)
        assert abs(r.lse[h] - float(torch.logsumexp(s, 0))) < 1e-13
        lo = n - len(w)
        assert np.allclose(r.weights[h, lo:n], w, atol=1e-14) and not r.weights[h, :lo].any() and not r.weights[h, n:].any()


def test_attend_closed_forms():
    k, v = np.zeros((2, 1, 4, 3)), np.arange(24.0).reshape(2, 1, 4, 3)
    q = np.ones((1, 3))
    r = paged.attend_row(q, k, v, [1, 0], 6, 1.0)
    assert np.allclose(r.out[0], np.concatenate([v[1, 0], v[0, 0, :2]]).mean(0)) and np.isclose(r.lse[0], np.log(6))
    assert paged.attend_row(q, k, v, [1, 0], 0, 1.0).lse[0] == -np.inf
    k[1, 0, 2, 0] = -np.inf                                      # that position has no weight
    assert np.allclose(paged.attend_row(q, k, v, [1], 4, 1.0).out[0], v[1, 0, [0, 1, 3]].mean(0))
    assert paged.attend_row(q, k, v, [1, 2], 5, 1.0).status == paged.STATUS_BAD_PAGE
    assert paged.attend_row(q, k, v, [1, 2], 4, 1.0).status == paged.STATUS_OK
    assert paged.attend_row(q, k, v, [1], 5, 1.0).status == paged.STATUS_BAD_LENGTH


def counts(tables, pages):
    c = [0] * pages
    for row in tables:
        for p in row:
            if p >= 0:
                c[p] += 1
    return c


@pytest.mark.parametrize("seed", range(40))
def test_fork_and_compact_keep_the_invariants(seed):
    rng = np.random.default_rng(seed)
    pages, slots, seqs = int(rng.integers(4, 40)), int(rng.integers(1, 5)), int(rng.integers(1, 6))
    width = int(rng.integers(1, 7))
    table, lengths, refs = [[-1] * width for _ in range(seqs)], [0] * seqs, [0] * pages
    text = {p: [None] * slots for p in range(pages)}             # what each page holds
    names = [[] for _ in range(seqs)]                            # what each sequence should read
    token = 0
    for step in range(12):
        n = int(rng.integers(1, 6))
        parent = rng.integers(-1, len(lengths), n).tolist()
        new = rng.integers(0, 2 * slots, n).tolist()
        r = paged.fork(table, lengths, refs, parent, new, slots, width)
        for src, dst in r.copies:
            text[dst] = list(text[src])
        story = []
        for i, p in enumerate(parent):
            old = names[p] if p >= 0 else []
            if r.status[i] == paged.STATUS_OK:
                assert r.lengths[i] == len(old) + new[i]
            else:
                assert r.lengths[i] in (0, len(old))
            story.append(list(old[: r.lengths[i]]))
            for j in range(len(story[i]), r.lengths[i]):         # every sequence writes its own
                token += 1
                text[r.table[i][j // slots]][j % slots] = token
                story[i].append(token)
        table, lengths, refs, names = r.table, r.lengths, r.refs, story
        assert refs == counts(table, pages)
        if step % 4 == 3:
            c = paged.compact(table, lengths, refs, slots)
            for src, dst in c.moves:
                text[dst] = list(text[src])
            table, refs = c.table, c.refs
            assert refs == counts(table, pages) and all(x > 0 for x in refs[: c.count]) and not any(refs[c.count:])
            assert not any(c.status)
        for row, n, want in zip(table, lengths, names):
            assert [text[row[j // slots]][j % slots] for j in range(n)] == want


def test_fork_statuses():
    table, refs = [[0, 1], [2, -1], [9, -1]], [1, 1, 1, 0]
    r = paged.fork(table, [3, 1, 1], refs, [0, 0, 1, 2, 5, -1], [0, 0, 9, 0, 0, 1], 2, 2)
    # the second child of 0 takes the last free page; the third cannot grow past its table; 2's page does not exist
    assert r.status == [0, 0, paged.STATUS_BAD_LENGTH, paged.STATUS_BAD_PAGE, paged.STATUS_BAD_PARENT, paged.STATUS_NO_PAGE]
    assert r.table[:3] == [[0, 1], [0, 3], [2, -1]] and r.copies == [(1, 3)] and r.refs == [2, 1, 1, 1]


def test_copy_pairs():
    moves, st = paged.copy_pairs([0, 1, 2, 3, 4], [5, 6, 6, 9, 5], 8)
    assert moves == [(2, 6), (4, 5)] and st == [0, 0, 0, 7, 0]
    moves, st = paged.copy_pairs([0, 5], [5, 0], 8)              # a swap: each would read what the other writes
    assert moves == [] and st == [7, 7]
    assert paged.append([3, 5], [0, 2, 3], [[1, 0], [7, 2]], 2, 4, 3) == ([(0, 1, 1), (1, 0, 0)], [0, 8])


def test_copy_pairs_refused_beside_sound():
    for pairs, want, status in (
            ([(1, 6), (-1, 6)], [(1, 6)], [0, 7]),
            ([(1, 5), (5, 5)], [(1, 5)], [0, 7]),
            ([(1, 6), (2, 6), (-1, 6)], [(2, 6)], [0, 0, 7]),
            ([(2, 6), (7, 6), (3, 7)], [(2, 6), (3, 7)], [0, 7, 0]),
            ([(-1, 6), (-1, 6)], [], [7, 7])):
        source, target = zip(*pairs)
        assert paged.copy_pairs(source, target, 8) == (want, status)


@pytest.mark.parametrize("seed", range(30))
def test_copy_pairs_does_what_its_statuses_say(seed):
    """Every target of a pair with status 0 holds the page of the last such pair afterwards, and no other page changes."""
    rng = np.random.default_rng(seed)
    pages, n = int(rng.integers(2, 12)), int(rng.integers(1, 20))
    source, target = (rng.integers(-1, pages + 1, n).tolist() for _ in range(2))
    moves, status = paged.copy_pairs(source, target, pages)
    want = list(range(pages))
    for s, t, st in zip(source, target, status):
        if st == 0:
            want[t] = s
    got = list(range(pages))
    for s, t in moves:
        got[t] = s                                            # sources are never targets, so any order will do
    assert got == want and len({t for _, t in moves}) == len(moves)


def test_fork_children_without_needs():
    """Children that need no page are not refused for want of pages, whoever came before them."""
    r = paged.fork([[0, 1, -1], [2, -1, -1], [3, -1, -1]], [6, 4, 3], [1, 1, 1, 1, 0], [0, 1, 2, 0, -1, 2, 1], [0, 9, 1, 0, 0, 0, 0], 4, 5)
    assert r.status == [0, 10, 0, 10, 0, 10, 0] and r.lengths == [6, 4, 4, 0, 0, 0, 4]
    assert r.refs == counts(r.table, 5) and r.copies == []
    r = paged.fork([[0, 1]], [7], [1, 1], [0, -1, 5, 0], [1, 0, 0, -1], 4, 2)
    assert r.status == [0, 0, paged.STATUS_BAD_PARENT, paged.STATUS_BAD_LENGTH] and r.lengths == [8, 0, 0, 0]
