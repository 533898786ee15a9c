"""Refusals of the paged cache's entry points before any device work, and their workspace sizes (no GPU: the calls here end in
the argument checks)."""
import ctypes

import pytest

import top_select_gumbel_amd as ts

FAKE = 0x1000      # never dereferenced on these paths
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    return ts.load_library()


def call(f, a, **kw):
    a.update(kw)
    return f(*[ctypes.byref(x) if isinstance(x, ctypes.Structure) else x for x in a.values()], None)


def attend(lib, **kw):
    pages = ts._Paged(1 << 20, 4096, 1024, 64)
    return call(lib.ts_cache_attend, dict(
        q=FAKE, dtype=1, batch=3, q_heads=8, kv_heads=4, dim=32, q_b=256, q_h=32, k=pages, v=pages, pages=10, slots=16, table=FAKE,
        width=200, stride=200, lengths=FAKE, scale=0.1, window=0, out=1 << 22, o_b=256, o_h=32, lse=None, weights=None, w_dtype=0,
        w_slots=0, w_b=0, w_h=0, status=None, ws=FAKE, ws_bytes=BIG), **kw)


@pytest.mark.parametrize("kw,word", [
    (dict(dtype=3), "dtype"), (dict(dtype=-1), "dtype"), (dict(batch=-1), "batch"), (dict(kv_heads=0), "heads"), (dict(kv_heads=3), "heads"),
    (dict(q_heads=0), "heads"), (dict(q_heads=-4), "heads"), (dict(q_heads=1 << 17), "q_heads"), (dict(dim=0), "dim"), (dict(dim=257), "dim"),
    (dict(scale=0.0), "scale"), (dict(scale=-1.0), "scale"), (dict(scale=float("nan")), "scale"), (dict(scale=float("inf")), "scale"),
    (dict(window=-1), "window"), (dict(pages=-1), "pages"), (dict(pages=1 << 31), "pages"), (dict(slots=0), "page_slots"),
    (dict(width=-1), "table_width"), (dict(stride=199), "table_stride"), (dict(q=None), "NULL"), (dict(table=None), "NULL"),
    (dict(lengths=None), "NULL"), (dict(out=None), "NULL"), (dict(out=FAKE), "may not be q"), (dict(pages=0), "pages"), (dict(q=FAKE + 1), "aligned"),
    (dict(out=FAKE + 1), "aligned"), (dict(q_b=-1), "q:"), (dict(q_b=1 << 61), "q:"), (dict(o_h=31), "overlap"), (dict(o_b=255), "overlap"),
    (dict(o_b=-256), "overlap"), (dict(k=ts._Paged(None, 64, 64, 64)), "NULL"), (dict(k=None), "NULL"), (dict(v=None), "NULL"),
    (dict(k=ts._Paged(FAKE + 1, 64, 64, 64)), "aligned"), (dict(v=ts._Paged(FAKE, 64, 64, 63)), "aligned"),
    (dict(v=ts._Paged(FAKE, -64, 64, 64)), "strides"), (dict(v=ts._Paged(FAKE, 1 << 60, 64, 64)), "strides"),
    (dict(weights=FAKE, w_dtype=3, w_slots=8, w_b=64, w_h=8), "weights_dtype"), (dict(weights=FAKE), "weights_slots"),
    (dict(w_slots=8), "out_weights"), (dict(weights=FAKE + 2, w_slots=8, w_b=64, w_h=8), "aligned"),
    (dict(weights=FAKE, w_slots=8, w_b=64, w_h=7), "overlap"), (dict(weights=FAKE, w_slots=8, w_b=63, w_h=8), "overlap"),
    (dict(batch=1 << 24), "too large"), (dict(batch=1 << 62), "strides"),
])
def test_attend_refusals(lib, kw, word):
    assert attend(lib, **kw) == ts.TS_ERR_INVALID_ARG
    assert word in ts.ts_last_error()


def test_attend_workspace(lib):
    assert attend(lib, batch=0, q=None, table=None, lengths=None, out=None, ws=None, ws_bytes=0) == ts.TS_OK
    need = lib.ts_cache_attend_workspace(1, 3, 8, 4, 32, 200 * 16, 0)
    assert need > 0 and need % 256 == 0
    assert attend(lib, ws=None) == ts.TS_ERR_WORKSPACE
    assert attend(lib, ws=FAKE + 16) == ts.TS_ERR_WORKSPACE
    assert attend(lib, ws_bytes=need - 1) == ts.TS_ERR_WORKSPACE and "needs" in ts.ts_last_error()
    assert lib.ts_cache_attend_workspace(1, 3, 8, 4, 32, 200 * 16, 200 * 16) > need
    assert lib.ts_cache_attend_workspace(1, 3, 8, 4, 32, 100, 0) == 0      # short sequences need none
    assert attend(lib, width=6, stride=6, ws=None, ws_bytes=0, pages=0) == ts.TS_ERR_INVALID_ARG and "pages" in ts.ts_last_error()
    for bad in [(-1, 8, 4, 32, 9, 0), (1, 8, 3, 32, 9, 0), (1, 8, 0, 32, 9, 0), (1, 8, 4, 0, 9, 0), (1, 8, 4, 300, 9, 0), (1, 8, 4, 32, -1, 0),
                (1, 8, 4, 32, 9, -1), (1 << 62, 8, 4, 32, 9, 0)]:
        assert lib.ts_cache_attend_workspace(1, *bad) == 0
    assert lib.ts_cache_attend_workspace(3, 3, 8, 4, 32, 3200, 0) == 0


def append(lib, **kw):
    pages = ts._Paged(1 << 20, 4096, 1024, 64)
    return call(lib.ts_cache_append, dict(
        k_new=FAKE, v_new=FAKE, tokens=9, batch=3, heads=4, slot_bytes=64, k_t=256, k_h=64, v_t=256, v_h=64, offsets=FAKE, k=pages,
        v=pages, pages=10, slots=16, table=FAKE, width=20, stride=20, lengths=FAKE, status=None), **kw)


@pytest.mark.parametrize("kw,word", [
    (dict(tokens=-1), "tokens"), (dict(tokens=1 << 31), "tokens"), (dict(batch=-1), "batch"), (dict(batch=(1 << 22) + 1), "batch"),
    (dict(heads=0), "kv_heads"), (dict(slot_bytes=0), "slot_bytes"), (dict(slot_bytes=4097), "slot_bytes"), (dict(slots=0), "page_slots"),
    (dict(stride=19), "table_stride"), (dict(offsets=None), "NULL"), (dict(table=None), "NULL"), (dict(lengths=None), "NULL"),
    (dict(k_new=None), "NULL"), (dict(v_new=None), "NULL"), (dict(k_t=-1), "strides"), (dict(v_h=1 << 61), "strides"),
    (dict(k=None), "NULL"), (dict(v=ts._Paged(None, 0, 0, 0)), "NULL"), (dict(k=ts._Paged(FAKE, 4096, 1024, 63)), "share"),
    (dict(k=ts._Paged(FAKE, 4095, 1024, 64)), "share"), (dict(v=ts._Paged(FAKE, 4096, 0, 64)), "share"), (dict(v=ts._Paged(FAKE, -1, 0, 64)), "share"),
])
def test_append_refusals(lib, kw, word):
    assert append(lib, **kw) == ts.TS_ERR_INVALID_ARG
    assert word in ts.ts_last_error()


def pools(*p):
    return (ts._Pool * max(1, len(p)))(*p)


def fork(lib, **kw):
    return call(lib.ts_pages_fork, dict(
        table=FAKE, seqs=4, width=8, stride=8, lengths=FAKE, refs=FAKE, pages=50, slots=16, parent=FAKE, n_new=None, children=5,
        out_table=1 << 20, out_width=9, out_stride=9, out_lengths=FAKE, out_refs=FAKE, pools=pools(ts._Pool(FAKE, 64, 64)), n=1,
        status=None, ws=FAKE, ws_bytes=BIG), **kw)


@pytest.mark.parametrize("kw,word", [
    (dict(seqs=-1), "seqs"), (dict(seqs=(1 << 16) + 1), "seqs"), (dict(children=-1), "children"), (dict(pages=-1), "pages"),
    (dict(children=(1 << 16) + 1), "children"), (dict(slots=0), "page_slots"), (dict(stride=7), "table_stride"), (dict(out_stride=8), "table_stride"), (dict(out_width=-1), "table_width"),
    (dict(children=1 << 16, out_width=1 << 20, out_stride=1 << 20), "too large"), (dict(table=None), "NULL"), (dict(lengths=None), "NULL"),
    (dict(parent=None), "NULL"), (dict(out_table=None), "NULL"), (dict(out_lengths=None), "NULL"), (dict(refs=None), "NULL"),
    (dict(out_refs=None), "NULL"), (dict(out_table=FAKE), "may not be"), (dict(n=-1), "n_pools"), (dict(pools=None), "NULL"),
    (dict(pools=pools(ts._Pool(None, 64, 64))), "NULL"), (dict(pools=pools(ts._Pool(FAKE, 63, 64))), "page_stride"),
    (dict(pools=pools(ts._Pool(FAKE, 64, 0))), "page_bytes"), (dict(pools=pools(ts._Pool(FAKE, 1 << 60, 64))), "page_stride"),
])
def test_fork_refusals(lib, kw, word):
    assert fork(lib, **kw) == ts.TS_ERR_INVALID_ARG
    assert word in ts.ts_last_error()


def test_fork_workspace(lib):
    need = lib.ts_pages_fork_workspace(4, 5, 50)
    assert need > 0 and fork(lib, ws_bytes=need - 1) == ts.TS_ERR_WORKSPACE and "needs" in ts.ts_last_error()
    assert fork(lib, ws=None) == ts.TS_ERR_WORKSPACE and fork(lib, ws=FAKE + 1) == ts.TS_ERR_WORKSPACE
    assert lib.ts_pages_fork_workspace(-1, 5, 50) == 0 and lib.ts_pages_fork_workspace(4, 5, 1 << 31) == 0
    assert fork(lib, seqs=0, children=0, pages=0, n=0, table=None, ws=None) == ts.TS_OK


def compact(lib, **kw):
    return call(lib.ts_pages_compact, dict(
        table=FAKE, seqs=4, width=8, stride=8, lengths=FAKE, refs=FAKE, pages=50, slots=16, out_table=FAKE, out_stride=8, out_refs=FAKE,
        out_map=FAKE, count=None, pools=pools(ts._Pool(FAKE, 64, 64)), n=1, status=None, ws=FAKE, ws_bytes=BIG), **kw)


@pytest.mark.parametrize("kw,word", [
    (dict(seqs=-1), "seqs"), (dict(pages=-1), "pages"), (dict(pages=0), "pages"), (dict(slots=0), "page_slots"), (dict(stride=7), "table_stride"),
    (dict(pages=(1 << 24) + 1), "pages"), (dict(n=4097), "n_pools"),
    (dict(out_stride=7), "out_stride"), (dict(out_stride=9), "input's place"), (dict(table=None), "NULL"), (dict(out_table=None), "NULL"),
    (dict(lengths=None), "NULL"), (dict(refs=None), "NULL"), (dict(out_refs=None), "NULL"), (dict(out_map=None), "NULL"),
    (dict(pools=None), "NULL"), (dict(n=-1), "n_pools"), (dict(pools=pools(ts._Pool(FAKE, 63, 64))), "page_stride"),
])
def test_compact_refusals(lib, kw, word):
    assert compact(lib, **kw) == ts.TS_ERR_INVALID_ARG
    assert word in ts.ts_last_error()


def test_compact_workspace(lib):
    need = lib.ts_pages_compact_workspace(50)
    assert need > 0 and compact(lib, ws_bytes=need - 1) == ts.TS_ERR_WORKSPACE and compact(lib, ws=None) == ts.TS_ERR_WORKSPACE
    assert lib.ts_pages_compact_workspace(-1) == 0


@pytest.mark.parametrize("kw,word", [
    (dict(n=-1), "n ="), (dict(n=(1 << 16) + 1), "n ="), (dict(pages=-1), "pages"), (dict(source=None), "NULL"), (dict(target=None), "NULL"),
    (dict(np=-1), "n_pools"), (dict(pools=None), "NULL"), (dict(pools=pools(ts._Pool(FAKE, 63, 64))), "page_stride"),
])
def test_copy_refusals(lib, kw, word):
    a = dict(source=FAKE, target=FAKE, n=3, pages=50, pools=pools(ts._Pool(FAKE, 64, 64)), np=1, status=None)
    assert call(lib.ts_pages_copy, a, **kw) == ts.TS_ERR_INVALID_ARG
    assert word in ts.ts_last_error()


def test_empty_calls(lib):
    assert append(lib, batch=0, offsets=None, table=None, lengths=None) == ts.TS_OK
    assert lib.ts_pages_copy(None, None, 0, 50, pools(ts._Pool(FAKE, 64, 64)), 1, None, None) == ts.TS_OK
    for st, word in ((ts.TS_ROW_BAD_PAGE, "page"), (ts.TS_ROW_BAD_LENGTH, "length"), (ts.TS_ROW_BAD_PARENT, "parent"), (ts.TS_ROW_NO_PAGE, "free")):
        assert word in ts.ts_status_string(st)


def test_binding_refuses_host_tensors_and_bad_shapes():
    torch = pytest.importorskip("torch")
    i = torch.zeros(2, dtype=torch.int32)
    q, pages, table = torch.zeros(2, 4, 8), torch.zeros(5, 2, 4, 8), torch.zeros(2, 3, dtype=torch.int32)
    with pytest.raises(ts.TopSelectError):
        ts.ts_cache_attend(q, pages, pages, table, i)
    with pytest.raises(ts.TopSelectError):
        ts.ts_cache_append(q, q, i, pages, pages, table, i)
    with pytest.raises(ts.TopSelectError):
        ts.ts_pages_fork(table, i, i, i, 4)
    with pytest.raises(ts.TopSelectError):
        ts.ts_pages_compact(table, i, i, 4)
    with pytest.raises(ts.TopSelectError):
        ts.ts_pages_copy(i, i, [pages])
    with pytest.raises(ts.TopSelectError):
        ts.PagePools([pages])


def test_divisor_of_the_kernels():
    """j / d by one product, as the kernels take it (for the divisors' extremes, in whole numbers)."""
    import random
    rng = random.Random(0)
    for d in list(range(1, 70)) + [1025, (1 << 20) - 1, 1 << 20, (1 << 29) + 1, (1 << 30) - 1, 1 << 30] + [rng.randrange(1, 1 << 30) for _ in range(300)]:
        bits = (d - 1).bit_length()
        mul = ((1 << (31 + bits)) + d - 1) // d
        assert mul < 1 << 32
        for j in [0, 1, d - 1, d, d + 1, 2 * d - 1, (1 << 31) - 1, (1 << 31) // d * d - 1, (1 << 31) // d * d] + [rng.randrange(1 << 31) for _ in range(20)]:
            if 0 <= j < 1 << 31:
                assert (j * mul) >> (31 + bits) == j // d


def test_attend_weights_slots_limit(lib):
    """Sums of weights_slots and a workgroup's positions (4096 at most) stay below 2^31 up to the limit."""
    most = 0x7FFFF000
    assert most + 4096 - 1 < 1 << 31 and -(-most // 4096) * 4096 < 1 << 31
    call = dict(batch=1, q_heads=2, kv_heads=2, weights=1 << 30, w_dtype=1, w_b=1 << 40, w_h=1 << 32, ws=None)
    for slots in (most + 1, most + 4095, 0x7FFFFF00, 0x7FFFFF01, (1 << 32) + 8):
        assert attend(lib, w_slots=slots, **call) == ts.TS_ERR_INVALID_ARG and "large" in ts.ts_last_error()
        assert lib.ts_cache_attend_workspace(1, 1, 2, 2, 32, 3200, slots) == 0
    assert attend(lib, w_slots=most, **call) == ts.TS_ERR_WORKSPACE
    assert lib.ts_cache_attend_workspace(1, 1, 2, 2, 32, 3200, most) > 2 * most * 4


@pytest.mark.parametrize("kw,meets", [
    # q [3, 8, 32] in 16 bits from FAKE on, rows of 64 bytes; the strides are in elements
    (dict(out=FAKE + 2), True), (dict(out=FAKE + 1536 - 2), True), (dict(out=FAKE + 1536), False), (dict(out=FAKE - 1534), True),
    (dict(out=FAKE - 1536), False),
    # halves of one buffer [3, 2, 8, 32], and of [3, 8, 64]: side by side, or shifted by an element
    (dict(q_b=512, o_b=512, out=FAKE + 512), False), (dict(q_b=512, o_b=512, out=FAKE + 510), True),
    (dict(q_b=512, o_b=512, out=FAKE + 514), True), (dict(q_b=512, o_b=512, out=FAKE - 512), False), (dict(q_b=512, o_b=512, out=FAKE - 1024), True),
    (dict(q_b=512, q_h=64, o_b=512, o_h=64, out=FAKE + 64), False), (dict(q_b=512, q_h=64, o_b=512, o_h=64, out=FAKE + 62), True),
    (dict(q_b=512, q_h=64, o_b=512, o_h=64, out=FAKE - 64), False), (dict(q_b=512, q_h=64, o_b=512, o_h=64, out=FAKE + 66), True),
    # other strides: the output's heads first, between the queries' rows or onto one of them
    (dict(q_b=512, q_h=64, o_b=64, o_h=192, out=FAKE + 64), False), (dict(q_b=512, q_h=64, o_b=64, o_h=192, out=FAKE + 128), True),
    (dict(q_b=512, q_h=64, o_b=96, o_h=320, out=FAKE + 2752), True),
    # one sequence: its stride counts for nothing; queries shared by all
    (dict(batch=1, q_b=0, o_b=1, out=FAKE + 512), False), (dict(batch=1, q_b=1 << 30, o_b=1, out=FAKE + 510), True),
    (dict(q_b=0, out=FAKE + 512), False), (dict(q_b=0, out=FAKE + 510), True), (dict(q_b=0, q_h=0, out=FAKE + 64), False),
    (dict(q_b=0, q_h=0, out=FAKE + 62), True),
])
def test_attend_output_beside_the_queries(lib, kw, meets):
    """An output that shares memory with the queries is refused, one between them is not (the next check's error comes)."""
    a = dict(batch=3, q_b=256, q_h=32, o_b=256, o_h=32)
    a.update({k: v for k, v in kw.items() if k != "out"})

    def rows(at, b, h):
        return {at + 2 * (i * (b if a["batch"] > 1 else 0) + j * h) + 2 * d for i in range(a["batch"]) for j in range(8) for d in range(32)}
    assert bool(rows(FAKE, a["q_b"], a["q_h"]) & rows(kw["out"], a["o_b"], a["o_h"])) == meets     # the case is what it says
    got = attend(lib, ws=None, **kw)
    if meets:
        assert got == ts.TS_ERR_INVALID_ARG and "overlaps" in ts.ts_last_error()
    else:
        assert got == ts.TS_ERR_WORKSPACE


@pytest.mark.parametrize("seed", range(60))
def test_attend_output_beside_the_queries_at_random(lib, seed):
    import random
    rng = random.Random(seed)
    for _ in range(40):
        batch, hq, dim = rng.randint(1, 4), rng.randint(1, 5), rng.randint(1, 9)

        def strides(apart):
            inner, outer = rng.sample([(hq, "h"), (batch, "b")], 2)
            s = {inner[1]: dim + rng.choice([0, 0, 1, 7])}
            s[outer[1]] = s[inner[1]] * (inner[0] - 1) + dim + rng.choice([0, 0, 2, 9, 40])
            return s if apart or rng.random() < 0.7 else {"b": rng.randint(0, 30), "h": rng.randint(0, 30)}
        q, o, shift = strides(False), strides(True), rng.randint(-60, 60)
        at = FAKE + 2 * shift

        def rows(at, s):
            return {at + 2 * (i * s["b"] + j * s["h"] + d) for i in range(batch) for j in range(hq) for d in range(dim)}
        meets = bool(rows(FAKE, q) & rows(at, o))
        # 2000 slots a row: sequences that need a workspace, which is missing
        got = attend(lib, batch=batch, q_heads=hq, kv_heads=1, dim=dim, q_b=q["b"], q_h=q["h"], o_b=o["b"], o_h=o["h"], out=at, ws=None)
        assert got == (ts.TS_ERR_INVALID_ARG if meets else ts.TS_ERR_WORKSPACE), (seed, batch, hq, dim, q, o, shift, ts.ts_last_error())


def test_append_without_table_columns(lib):
    """A table of width 0 may be NULL, as for the other calls: nothing is read of it (the slots that share memory come next)."""
    bad = ts._Paged(FAKE, 4096, 1024, 63)
    assert append(lib, table=None, width=0, stride=0, k=bad) == ts.TS_ERR_INVALID_ARG and "share" in ts.ts_last_error()
    assert append(lib, table=None, width=1, stride=1, k=bad) == ts.TS_ERR_INVALID_ARG and "NULL" in ts.ts_last_error()
