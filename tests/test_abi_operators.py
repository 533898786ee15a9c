"""Refusals of ts_token_logp, ts_token_logp_backward and ts_cache_evict before any device work, and their workspace
sizes (no GPU: the calls here end in the argument checks)."""
import ctypes

import pytest

import top_select_gumbel_amd as ts

FAKE = 0x1000      # never dereferenced on these paths
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    return ts.load_library()


def logp(lib, **kw):
    a = dict(logits=FAKE, dtype=0, rows=2, vocab=10000, stride=10000, tokens=FAKE, t=None, n_top=0, logp=FAKE, rank=FAKE,
             entropy=FAKE, lse=FAKE, idx=None, top=None, stats=FAKE, status=FAKE, ws=FAKE, ws_bytes=BIG)
    a.update(kw)
    return lib.ts_token_logp(*a.values(), None)


@pytest.mark.parametrize("kw,word", [
    (dict(rows=-1), "rows"), (dict(vocab=0), "vocab"), (dict(vocab=(1 << 30) + 1, stride=1 << 31), "vocab"),
    (dict(stride=9999), "stride"), (dict(dtype=3), "dtype"), (dict(dtype=-1), "dtype"), (dict(logits=None), "NULL"),
    (dict(logits=FAKE + 2), "aligned"), (dict(logits=FAKE + 1, dtype=1), "aligned"), (dict(n_top=-1), "n_top"),
    (dict(n_top=65), "n_top"), (dict(tokens=None), "tokens"), (dict(n_top=3), "out_top_idx"), (dict(n_top=3, idx=FAKE), "out_top_idx"),
    (dict(stats=FAKE + 8), "aligned"), (dict(rows=1 << 24), "too large"),
])
def test_logp_refusals(lib, kw, word):
    assert logp(lib, **kw) == ts.TS_ERR_INVALID_ARG
    assert word in ts.ts_last_error()


def test_logp_workspace(lib):
    assert logp(lib, ws=None) == ts.TS_ERR_WORKSPACE
    assert logp(lib, ws=FAKE + 16) == ts.TS_ERR_WORKSPACE and "aligned" in ts.ts_last_error()
    need = ts.ts_workspace_bytes(ts.TS_OP_TOKEN_LOGP, 2, 10000, 0)
    assert need > 0 and need % 256 == 0
    assert logp(lib, ws_bytes=need - 1) == ts.TS_ERR_WORKSPACE and "needs" in ts.ts_last_error()
    assert ts.ts_workspace_bytes(ts.TS_OP_TOKEN_LOGP, 2, 10000, 20) > need
    for rows, vocab, n in [(-1, 10, 0), (1, 0, 0), (1, (1 << 30) + 1, 0), (1, 10, -1), (1, 10, 65)]:
        assert ts.ts_workspace_bytes(ts.TS_OP_TOKEN_LOGP, rows, vocab, n) == 0
    # no row: nothing is needed; a bad shape is still refused
    assert logp(lib, rows=0, logits=None, tokens=None, ws=None, ws_bytes=0) == ts.TS_OK
    assert logp(lib, rows=0, vocab=0) == ts.TS_ERR_INVALID_ARG


def backward(lib, **kw):
    a = dict(logits=1 << 20, dtype=0, rows=2, vocab=100, stride=100, tokens=FAKE, t=None, stats=FAKE, a=FAKE, h=None, l=None,
             out=1 << 24, out_stride=100)
    a.update(kw)
    return lib.ts_token_logp_backward(*a.values(), None)


@pytest.mark.parametrize("kw,word", [
    (dict(rows=-1), "rows"), (dict(vocab=0), "vocab"), (dict(stride=99), "stride"), (dict(dtype=7), "dtype"),
    (dict(logits=None), "NULL"), (dict(out_stride=99), "grad_stride"), (dict(stats=None), "stats"), (dict(out=None), "required"),
    (dict(tokens=None), "tokens"), (dict(stats=FAKE + 4), "aligned"), (dict(out=(1 << 24) + 2), "aligned"),
    (dict(out=(1 << 20) + 4), "overlap"), (dict(out=1 << 20, out_stride=101), "overlap"), (dict(out=(1 << 20) + 400), "overlap"),
])
def test_backward_refusals(lib, kw, word):
    assert backward(lib, **kw) == ts.TS_ERR_INVALID_ARG
    assert word in ts.ts_last_error()


def test_backward_empty_batch(lib):
    assert backward(lib, rows=0, logits=None, stats=None, out=None, tokens=None, a=None) == ts.TS_OK


def evict(lib, **kw):
    cache = ts._Cache(1 << 20, 4096, 1024, 64, 64)
    a = dict(score=FAKE, rows=4, slots=16, score_stride=16, position=FAKE, position_stride=16, lengths=FAKE, keep=FAKE, keep_max=8,
             weights=FAKE, dtype=0, n=2, w_row=32, w_stride=16, sinks=1, recent=1, out_score=1 << 22, os=8, out_position=1 << 23,
             op=8, out_lengths=FAKE, source=FAKE, status=None, k=cache, v=None, heads=2, ws=FAKE, ws_bytes=BIG)
    a.update(kw)
    for c in "kv":
        if a[c] is not None:
            a[c] = ctypes.byref(a[c])
    return lib.ts_cache_evict(*a.values(), None)


@pytest.mark.parametrize("kw,word", [
    (dict(rows=-1), "rows"), (dict(slots=0), "slots"), (dict(score_stride=15), "score_stride"), (dict(position_stride=15), "position_stride"),
    (dict(keep_max=0), "keep_max"), (dict(os=7), "out_score_stride"), (dict(op=7), "out_position_stride"), (dict(sinks=-1), "sinks"),
    (dict(recent=-1), "recent"), (dict(n=-1), "n_weights"), (dict(dtype=9), "weights_dtype"), (dict(w_stride=-1), "stride"),
    (dict(w_row=-1), "stride"), (dict(heads=0), "heads"), (dict(heads=3), "heads"), (dict(score=None), "required"),
    (dict(position=None), "required"), (dict(lengths=None), "required"), (dict(keep=None), "required"),
    (dict(out_score=None), "required"), (dict(out_position=None), "required"), (dict(out_lengths=None), "required"),
    (dict(source=None), "required"), (dict(out_score=FAKE), "input's place"), (dict(out_position=FAKE), "input's place"),
    (dict(weights=None), "NULL"), (dict(weights=FAKE + 2), "aligned"), (dict(k=ts._Cache(None, 0, 0, 64, 64)), "NULL"),
    (dict(k=ts._Cache(FAKE, 0, 0, 63, 64)), "slot_stride"), (dict(v=ts._Cache(FAKE, 0, 0, 64, 0)), "slot_bytes"),
    (dict(v=ts._Cache(FAKE, -1, 0, 64, 64)), "negative"), (dict(rows=1 << 24), "too large"),
])
def test_evict_refusals(lib, kw, word):
    assert evict(lib, **kw) == ts.TS_ERR_INVALID_ARG
    assert word in ts.ts_last_error()


def test_evict_workspace(lib):
    assert evict(lib, ws=None) == ts.TS_ERR_WORKSPACE
    assert evict(lib, ws=FAKE + 16) == ts.TS_ERR_WORKSPACE
    need = ts.ts_workspace_bytes(ts.TS_OP_CACHE_EVICT, 4, 16, 8)
    assert need > 0 and evict(lib, ws_bytes=need - 1) == ts.TS_ERR_WORKSPACE and "needs" in ts.ts_last_error()
    assert evict(lib, rows=0, score=None, position=None, lengths=None, keep=None, ws=None) == ts.TS_OK
    for rows, slots, keep in [(-1, 4, 4), (1, 0, 4), (1, 4, 0)]:
        assert ts.ts_workspace_bytes(ts.TS_OP_CACHE_EVICT, rows, slots, keep) == 0


def test_status_string():
    assert "token" in ts.ts_status_string(ts.TS_ROW_BAD_TOKEN)


def test_binding_refuses_host_tensors():
    torch = pytest.importorskip("torch")
    x = torch.zeros(2, 8)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ts.TopSelectError):
        ts.ts_token_logp(x, i)
    with pytest.raises(ts.TopSelectError):
        ts.ts_token_logp_backward(x, i, None, torch.zeros(2, 4))
    with pytest.raises(ts.TopSelectError):
        ts.ts_cache_evict(x, torch.zeros(2, 8, dtype=torch.int32), i, i, 4)


@pytest.mark.parametrize("rows,vocab", [((1 << 47) + 1, 1 << 30), (1 << 62, 2), ((1 << 63) - 1, 1), ((1 << 61) + 1, 3 * 8192)])
def test_row_counts_whose_products_wrap(lib, rows, vocab):
    # rows x tiles (and rows x stride) of these are small or negative numbers in 64 bits
    assert ts.ts_workspace_bytes(ts.TS_OP_TOKEN_LOGP, rows, vocab, 0) == 0
    assert logp(lib, rows=rows, vocab=vocab, stride=vocab) == ts.TS_ERR_INVALID_ARG and "too large" in ts.ts_last_error()
    assert backward(lib, rows=rows, vocab=vocab, stride=vocab, out_stride=vocab) == ts.TS_ERR_INVALID_ARG
    assert "too large" in ts.ts_last_error()


def test_strides_whose_products_wrap(lib):
    assert logp(lib, rows=1 << 10, stride=1 << 60) == ts.TS_ERR_INVALID_ARG and "too large" in ts.ts_last_error()
    for kw in (dict(stride=1 << 60), dict(out_stride=1 << 60)):
        assert backward(lib, rows=1 << 10, **kw) == ts.TS_ERR_INVALID_ARG and "too large" in ts.ts_last_error()


@pytest.mark.parametrize("offset", [0, 4, -4, 396, -396, 800 - 396, -800, 800 + 4, 3 * 800])
def test_interleaved_gradient_rows_that_share_elements(lib, offset):
    # rows of 400 bytes, 800 apart: from 400 to 400 bytes beside each other they are apart (offsets 400, -400, 1200 ...)
    kw = dict(rows=5, vocab=100, stride=200, out=(1 << 20) + offset, out_stride=200)
    if offset == 0:      # taking the logits' place is allowed, but not one row short
        kw["out_stride"] = 199
    assert backward(lib, **kw) == ts.TS_ERR_INVALID_ARG and "overlap" in ts.ts_last_error()
