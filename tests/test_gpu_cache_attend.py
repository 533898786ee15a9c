"""GPU tests of ts_cache_attend against the binary64 oracle over the stored values.

Tolerances, with u = 2^-24. A score is a dot product of exact fp32 products (fp32 inputs: one rounding each), added in fp32 by
units that may cut off instead of rounding: |ds_j| <= 2 (dim + 1) u sum_i |q_i k_ij|. Relative to the largest, p_j =
exp(scale (s_j - m)) then is off by scale |ds_j| + 3 u scale |s_j - m| (difference, product, constant) + 2^-21 (the hardware's
exponential) and, for every time the running maximum grew, which is at most once a tile of a wave and once a part, 2^-21 and
its share of the exponent, which adds up to the 3 u term once more. The largest of these is off for the sum S too, whose
terms are added one after the other in a lane's tiles, then over lanes, waves and parts: (n / 16 + 64) u more. The weighted
values are added in fp32 by the matrix units (two products a tile): 2 u (n / 2 + 64) of the sum of |w v|; P in two 16-bit parts
loses 2^-16 (bf16) or 2^-21 (fp16). Last comes a half step of the output's type. The hardware's exponential gives 0 below fp32's
smallest normal number: p_j < 2^-126 counts as 0, which S >= 1 (the largest's own term) makes an error of at most 2^-126 in a weight.
"""
import numpy as np
import pytest

from oracle import paged
import top_select_gumbel_amd as ts
from gpu_helpers import banner, host, torch_cuda

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
FLUSHED = 2.0 ** -126
HALF = {"float32": 2.0 ** -24, "bfloat16": 2.0 ** -8, "float16": 2.0 ** -11}
TINY = {"float32": 2.0 ** -149, "bfloat16": 2.0 ** -133, "float16": 2.0 ** -25}
P_LOSS = {"float32": 0.0, "bfloat16": 2.0 ** -16, "float16": 2.0 ** -21}


def compare(r, got_out, got_lse, got_w, scale, dtype, wtype, group, label):
    """One sequence's outputs against the oracle's row within the bounds above."""
    if r.status != paged.STATUS_OK:
        assert np.isnan(got_out).all(), label
        assert got_lse is None or np.isnan(got_lse).all(), label
        assert got_w is None or np.isnan(got_w).all(), label
        return
    if r.scores is None:
        assert not got_out.any() and (got_lse is None or (got_lse == -np.inf).all()) and (got_w is None or not got_w.any()), label
        return
    n = r.scores.shape[1]
    for h in range(len(r.lse)):
        if r.lse[h] == -np.inf:
            assert not got_out[h].any() and (got_lse is None or got_lse[h] == -np.inf) and (got_w is None or not got_w[h].any()), label
            continue
        s, a = r.scores[h], r.magnitude[h]
        live = np.isfinite(s)
        m, dim = s[live].max(), r.values.shape[2]
        ds = np.where(live, 2 * (dim + 1) * U * np.where(live, a, 0.0), 0.0)
        d = np.where(live, scale * ds + 6 * U * scale * np.where(live, m - s, 0.0) + 2.0 ** -21 * (n / 64 + 8), 0.0)
        seen = live & (scale * (m - np.where(live, s, m)) < 88.0)   # beyond, e^-88 < 2^-126
        d = np.where(seen, d, 0.0)
        total = d.max() + (n / 16 + 64) * U
        w = np.where(live, np.exp(scale * (np.where(live, s, m) - m)), 0.0)
        w /= w.sum()
        v = np.abs(r.values[h // group])
        tol = ((d + total + P_LOSS[dtype] + 2 * U * (n / 2 + 64)) * w) @ v
        tol = tol * 1.01 + HALF[dtype] * np.abs(r.out[h]) * 1.01 + TINY[dtype] + FLUSHED * v.sum(0)
        err = np.abs(got_out[h] - r.out[h])
        assert (err <= tol).all(), f"{label} head {h}: out off by {err.max():.3g}, allowed {tol[err.argmax()]:.3g}"
        if got_lse is not None:
            t = scale * ds.max() + total + 4 * U * (abs(r.lse[h]) + abs(scale * m) + abs(r.lse[h] - scale * m) + 1)
            assert abs(got_lse[h] - r.lse[h]) <= t, f"{label} head {h}: lse {got_lse[h]} for {r.lse[h]}, allowed {t:.3g}"
        if got_w is not None:
            full = np.zeros_like(r.weights[h])
            full[:] = HALF[wtype] * r.weights[h] * 1.01 + TINY[wtype] + FLUSHED
            start = r.start
            full[start:start + n] += (d + total) * r.weights[h, start:start + n] * 1.01
            err = np.abs(got_w[h] - r.weights[h])
            assert (err <= full).all(), f"{label} head {h}: weight off by {err.max():.3g}, allowed {full[(err - full).argmax()]:.3g}, at {(err - full).argmax()}"


def check(batch=2, hq=4, hk=2, dim=64, n=100, slots=16, dtype="bfloat16", lengths=None, window=0, wtype=None, scale=None, seed=0,
          slots_first=False, spread=1.0, edit=None, wide=0, extra=3, stale=float("nan")):
    torch = torch_cuda()
    lengths = np.full(batch, n, np.int32) if lengths is None else np.asarray(lengths, np.int32)
    batch, top = len(lengths), max(1, int(max(lengths)))
    width = -(-top // slots)
    pages = batch * width + extra
    banner(f"attend {dtype} b={batch} hq={hq} hk={hk} dim={dim} n={lengths[:6].tolist()} slots={slots} window={window} weights={wtype}")
    gen = torch.Generator().manual_seed(seed)
    t = getattr(torch, dtype)
    shape = (pages, slots, hk, dim + wide) if slots_first else (pages, hk, slots, dim + wide)
    k, v = (torch.randn(shape, generator=gen).to(t) for _ in range(2))
    if slots_first:
        k, v = k.transpose(1, 2), v.transpose(1, 2)
    q = (torch.randn((batch, hq, dim + wide), generator=gen) * spread).to(t)[..., :dim]
    table = torch.randperm(pages, generator=gen)[: batch * width].view(batch, width).to(torch.int32)
    held = torch.from_numpy(-(-lengths.clip(0) // slots))
    lo = np.maximum(0, lengths - window) if window else np.zeros_like(lengths)
    # what is not attended holds anything: slots past the end, before the window, pages of no one, table entries past the end
    attended = torch.zeros((pages, slots), dtype=torch.bool)
    for b in range(batch):
        for j in range(int(lo[b]), int(lengths[b])):
            attended[table[b, j // slots], j % slots] = True
    k.transpose(1, 2)[~attended] = stale
    v.transpose(1, 2)[~attended] = stale
    if wide:
        k[..., dim:], v[..., dim:] = stale, stale
    table[torch.arange(width)[None, :] >= held[:, None]] = -7
    for b in range(batch):
        table[b, : int(lo[b]) // slots] = 1 << 30                      # freed behind the window
    kd, vd = k[..., :dim], v[..., :dim]
    if edit is not None:
        edit(q, kd, vd, table, lengths)
    scale = dim ** -0.5 if scale is None else scale
    dev = [x.cuda() for x in (q, k, v)]
    r = ts.ts_cache_attend(dev[0], dev[1][..., :dim], dev[2][..., :dim], table.cuda(), torch.from_numpy(lengths).cuda(), scale=scale,
                           window=window, weights_slots=top if wtype else 0, weights_dtype=getattr(torch, wtype) if wtype else None)
    torch.cuda.synchronize()
    out, lse = host(r.out.double()), host(r.lse.double())
    w = host(r.weights.double()) if wtype else None
    q64, k64, v64 = (x.double().numpy() for x in (q, kd, vd))
    s32 = float(np.float32(scale))
    for b in range(batch):
        o = paged.attend_row(q64[b], k64, v64, table[b].tolist(), int(lengths[b]), s32, window, top if wtype else 0)
        o.start = int(lo[b])
        assert int(r.status[b]) == o.status, f"sequence {b}: status {int(r.status[b])} for {o.status}"
        compare(o, out[b], lse[b], None if w is None else w[b], s32, dtype, wtype, hq // hk, f"sequence {b}")
    return r


TYPES = ["float32", "bfloat16", "float16"]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 32, 33, 63, 129, 256, 257, 600])
def test_lengths(dtype, n):
    check(n=n, dtype=dtype, wtype=dtype, seed=n)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim", [1, 7, 8, 33, 64, 72, 80, 96, 127, 128, 136, 200, 255, 256])
def test_dims(dtype, dim):
    check(dim=dim, n=333, dtype=dtype, seed=dim, lengths=[333, 40])


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("slots", [1, 3, 15, 16, 24, 32, 48, 300, 1025])
def test_page_sizes(dtype, slots):
    check(n=500, slots=slots, dtype=dtype, lengths=[500, 37, 299, 1], seed=slots)


@pytest.mark.parametrize("hq,hk", [(1, 1), (5, 5), (6, 2), (7, 1), (15, 1), (16, 1), (17, 1), (32, 2), (40, 1), (70, 2)])
@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
def test_heads(hq, hk, dtype):
    check(hq=hq, hk=hk, n=290, dtype=dtype, lengths=[290, 77], wtype="float32", seed=hq)


@pytest.mark.parametrize("window", [1, 5, 16, 31, 100, 299, 300, 1000])
@pytest.mark.parametrize("slots", [16, 24])
def test_windows(window, slots):
    check(n=300, window=window, slots=slots, lengths=[300, 299, 17, 0, 160], wtype="float16", dtype="float16", seed=window)


@pytest.mark.parametrize("dtype", TYPES)
def test_ragged_batches_with_empty_sequences(dtype):
    rng = np.random.default_rng(3)
    lengths = rng.integers(0, 700, 37)
    lengths[[0, 5, 6, 36]] = 0
    lengths[9], lengths[10] = 3000, 1
    check(lengths=lengths, dtype=dtype, wtype="float32", hk=1, hq=3)
    check(lengths=[0, 0, 0], dtype=dtype, wtype="float32")


def test_more_sequences_than_threads():
    rng = np.random.default_rng(4)
    check(lengths=rng.integers(0, 40, 700), hq=2, hk=1, slots=8, dim=16, dtype="float16")
    check(lengths=np.r_[rng.integers(0, 20, 600), 4000, rng.integers(0, 20, 100)], hq=2, hk=1, slots=80, dim=16, dtype="float16")


@pytest.mark.parametrize("dtype", TYPES)
def test_few_long_sequences(dtype):
    check(lengths=[9001, 4097], hq=2, hk=1, dtype=dtype, dim=64, wtype="bfloat16")
    check(lengths=[20000], hq=4, hk=4, dtype=dtype, dim=128, window=15000)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("slots_first,wide", [(True, 0), (False, 3), (True, 5)])
def test_layouts(dtype, slots_first, wide):
    check(n=280, dtype=dtype, slots_first=slots_first, wide=wide, dim=96, wtype=dtype)
    check(n=280, dtype=dtype, slots_first=slots_first, wide=wide, dim=33)


@pytest.mark.parametrize("dtype", TYPES)
def test_peaked_and_far_scores(dtype):
    # a few positions take all weight; others lie hundreds of octaves below
    check(n=400, dtype=dtype, spread=8.0, scale=1.0, dim=128, wtype="float32")
    check(n=400, dtype=dtype, spread=1.0, scale=2.0 ** -20, dim=128, wtype="float32")
    check(n=400, dtype=dtype, spread=4.0, scale=30.0, dim=32, wtype="float32")


def test_many_small_weights_beside_a_large_one():
    """fp16's P: 8000 positions of weight e^-11 of the largest each, 13% of the sum together, are not lost."""
    def edit(q, k, v, table, lengths):
        k.zero_(), v.fill_(1.0)
        q.zero_()
        q[..., 0] = 1.0
        k[..., 0] = -11.0
        k[table[0, 3], :, 5, 0] = 0.0
        v[table[0, 3], :, 5] = 0.0
    for dtype in ("float16", "bfloat16"):
        r = check(lengths=[8000], slots=16, hq=2, hk=1, dtype=dtype, scale=1.0, edit=edit, wtype="float32", stale=0.0)
        want = 7999 * np.exp(-11) / (1 + 7999 * np.exp(-11))
        assert abs(float(r.out[0, 0, 0]) / want - 1) < 2.0 ** -8


@pytest.mark.parametrize("dtype", TYPES)
def test_infinities_and_nan(dtype):
    torch = torch_cuda()

    def masked(q, k, v, table, lengths):      # -inf scores: no weight; sequence 1 as a whole
        q[..., 0] = 1.0
        k[table[0, 1], :, 3, 0] = -float("inf")
        k[table[1], :, :, 0] = -float("inf")
    for n in (40, 400):
        r = check(lengths=[n, 37], dtype=dtype, edit=masked, wtype="float32", stale=0.0)
        assert float(r.lse[1, 0]) == -np.inf and not bool(r.out[1].any())
    lowest = float(torch.finfo(getattr(torch, dtype)).min)

    def low(q, k, v, table, lengths):         # a mask of the type's lowest value, through a dim of its own
        q[..., 0] = 1.0
        k[..., 0] = 0.0
        k[table[0, 0], :, 2:9, 0] = lowest
    check(lengths=[100, 290], dtype=dtype, edit=low, scale=1.0, wtype="float32", stale=0.0)
    # NaN in an attended key or value shows in its heads, in its sequence only
    x = check(lengths=[300, 300, 300], dtype=dtype)
    k, v = (torch.randn(60, 2, 16, 64, device="cuda").to(getattr(torch, dtype)) for _ in range(2))
    table = torch.arange(57, dtype=torch.int32, device="cuda").view(3, 19)
    q, ln = torch.randn(3, 4, 64, device="cuda").to(k.dtype), torch.full((3,), 300, dtype=torch.int32, device="cuda")
    k[table[0, 4].long(), 1, 3, 5] = float("nan")
    v[table[2, 18].long(), 0, 11, 7] = float("inf")
    r = ts.ts_cache_attend(q, k, v, table, ln)
    out = host(r.out.double())
    assert np.isnan(out[0, 2:]).all() and np.isfinite(out[0, :2]).all() and np.isfinite(out[1]).all()
    assert not np.isfinite(out[2, :2, 7]).any() and np.isfinite(out[2, 2:]).all() and not host(r.status).any()
    assert not host(x.status).any()


@pytest.mark.parametrize("n", [100, 900])
def test_bad_pages_and_lengths(n):
    def edit(q, k, v, table, lengths):
        table[1, 2], table[2, 0], table[5, (n - 1) // 16] = 1 << 30, -1, k.shape[0]
        lengths[3], lengths[4] = -1, table.shape[1] * 16 + 1
    r = check(lengths=[n] * 7, dtype="bfloat16", edit=edit, wtype="float32")
    assert host(r.status).tolist() == [0, 7, 7, 8, 8, 7, 0]
    torch = torch_cuda()
    # a length above weights_slots is refused for the sequence
    q, k = torch.randn(2, 2, 32, device="cuda"), torch.randn(40, 1, 16, 32, device="cuda")
    table = torch.arange(40, dtype=torch.int32, device="cuda").view(2, 20)
    r = ts.ts_cache_attend(q, k, k, table, torch.tensor([50, 30], dtype=torch.int32, device="cuda"), weights_slots=40)
    assert host(r.status).tolist() == [8, 0] and bool(r.weights[0].isnan().all()) and bool(r.weights[1].isfinite().all())


def plain_call(seed=0, batch=3, n=700, dtype="bfloat16", device="cuda"):
    torch = torch_cuda()
    gen = torch.Generator(device=device).manual_seed(seed)
    t = getattr(torch, dtype)
    width = -(-n // 16)
    k, v = (torch.randn((batch * width, 2, 16, 64), generator=gen, device=device).to(t) for _ in range(2))
    q = torch.randn((batch, 6, 64), generator=gen, device=device).to(t)
    table = torch.randperm(batch * width, generator=gen, device=device).view(batch, width).to(torch.int32)
    lengths = torch.randint(1, n, (batch,), generator=gen, device=device).to(torch.int32)
    return dict(q=q, k_pages=k, v_pages=v, table=table, lengths=lengths, weights_slots=n, weights_dtype=torch.float32)


def equal(a, b):
    torch = torch_cuda()
    return all(torch.equal(x, y) for x, y in zip(a, b) if x is not None)


def test_same_bits_every_time_and_outputs_given():
    torch = torch_cuda()
    banner("attend: determinism, out given, rows behind the batch untouched")
    a = plain_call()
    first = ts.ts_cache_attend(**a)
    for _ in range(3):
        assert equal(first, ts.ts_cache_attend(**a))
    buf = torch.full((5, 9, 80), 7.0, dtype=a["q"].dtype, device="cuda")
    out = buf[:3, 1:7, 8:72]
    r = ts.ts_cache_attend(out=out, **a)
    assert r.out.data_ptr() == out.data_ptr() and equal(first, r)
    untouched = torch.ones_like(buf, dtype=torch.bool)
    untouched[:3, 1:7, 8:72] = False
    assert bool((buf[untouched] == 7.0).all())
    none = ts.ts_cache_attend(a["q"], a["k_pages"], a["v_pages"], a["table"], a["lengths"], want_lse=False)
    assert none.lse is None and none.weights is None and torch.equal(none.out, first.out)


def test_captured_and_replayed():
    """Two calls in one graph and the same in another, replayed in turn with eager calls between."""
    torch = torch_cuda()
    banner("attend: graphs")
    calls = [plain_call(s, n=n) for s, n in ((1, 900), (2, 200))]
    want = [ts.ts_cache_attend(**c) for c in calls]
    torch.cuda.synchronize()
    graphs, got = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got.append([ts.ts_cache_attend(**c) for c in calls])
        graphs.append(g)
    other = torch.cuda.Stream()
    for turn in range(4):
        for r in got:
            for x in r:
                x.out.fill_(3.0), x.lse.fill_(3.0), x.weights.fill_(3.0)
        torch.cuda.synchronize()
        graphs[0].replay()
        with torch.cuda.stream(other):
            graphs[1].replay()
            eager = ts.ts_cache_attend(**calls[0])
        torch.cuda.synchronize()
        for r in got:
            assert all(equal(x, y) for x, y in zip(r, want)), turn
        assert equal(eager, want[0])
        # the graph reads what its inputs hold now
        calls[0]["q"].mul_(-1)
        want = [ts.ts_cache_attend(**c) for c in calls]


def test_side_stream_and_two_calls_at_once():
    torch = torch_cuda()
    banner("attend: streams")
    a, b = plain_call(5, n=2000), plain_call(6, n=3000)
    want = [ts.ts_cache_attend(**a), ts.ts_cache_attend(**b)]
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        with torch.cuda.stream(s1):
            x = ts.ts_cache_attend(**a)
        with torch.cuda.stream(s2):
            y = ts.ts_cache_attend(**b)
        torch.cuda.synchronize()
        assert equal(x, want[0]) and equal(y, want[1])


def test_empty_batch():
    torch = torch_cuda()
    k = torch.randn(4, 1, 16, 32, device="cuda")
    r = ts.ts_cache_attend(k.new_empty(0, 2, 32), k, k, torch.empty(0, 3, dtype=torch.int32, device="cuda"),
                           torch.empty(0, dtype=torch.int32, device="cuda"), weights_slots=5)
    assert r.out.shape == (0, 2, 32) and r.lse.shape == (0, 2) and r.weights.shape == (0, 2, 5)
    z = torch.zeros(2, dtype=torch.int32, device="cuda")
    r = ts.ts_cache_attend(k.new_ones(2, 2, 32), k, k, torch.empty(2, 0, dtype=torch.int32, device="cuda"), z)
    assert not bool(r.out.any()) and bool((r.lse == -np.inf).all()) and not host(r.status).any()


def test_offsets_past_32_bits():
    """Pages more than 4 GB into the cache, and a table of a sequence that uses the first and the last one."""
    torch = torch_cuda()
    banner("attend: 5 GB of keys")
    pages, dim = 160_000, 128
    k = torch.empty(pages, 1, 128, dim, dtype=torch.bfloat16, device="cuda")
    v = torch.empty(pages, 1, 128, dim, dtype=torch.bfloat16, device="cuda")
    ids = torch.tensor([pages - 1, 0, 131_072, 65_536, 77], device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(1)
    small = [torch.randn((5, 1, 128, dim), generator=gen, device="cuda").to(torch.bfloat16) for _ in range(2)]
    k[ids], v[ids] = small[0], small[1]
    q = torch.randn((1, 4, dim), generator=gen, device="cuda").to(torch.bfloat16)
    n = torch.tensor([600], dtype=torch.int32, device="cuda")
    r = ts.ts_cache_attend(q, k, v, ids.to(torch.int32).view(1, 5), n)
    near = ts.ts_cache_attend(q, *small, torch.arange(5, dtype=torch.int32, device="cuda").view(1, 5), n)
    assert equal(r, near) and not host(r.status).any()


def test_views_of_queries_tables_and_outputs():
    """Queries shared by all sequences (stride 0) or heads first in memory, a table whose rows lie apart, outputs heads first."""
    torch = torch_cuda()
    a = plain_call(9)
    want = ts.ts_cache_attend(**a)
    heads_first = a["q"].transpose(0, 1).contiguous().transpose(0, 1)
    table = torch.full((3, 99), -5, dtype=torch.int32, device="cuda")[:, : a["table"].shape[1]].copy_(a["table"])
    out = torch.empty(6, 3, 64, dtype=a["q"].dtype, device="cuda").transpose(0, 1)
    r = ts.ts_cache_attend(**{**a, "q": heads_first, "table": table}, out=out)
    assert r.out.data_ptr() == out.data_ptr() and equal(r, want)
    one = a["q"][:1].expand(3, 6, 64)
    assert equal(ts.ts_cache_attend(**{**a, "q": one}), ts.ts_cache_attend(**{**a, "q": one.contiguous()}))
    # keys and values that share memory: read only
    shared = ts.ts_cache_attend(**{**a, "v_pages": a["k_pages"]})
    assert equal(shared, ts.ts_cache_attend(**{**a, "v_pages": a["k_pages"].clone()}))
    # the same pages in two sequences' tables
    both = a["table"][:1].expand(3, -1).contiguous()
    n = torch.full((3,), int(a["lengths"][0]), dtype=torch.int32, device="cuda")
    r = ts.ts_cache_attend(**{**a, "table": both, "lengths": n, "q": one})
    assert float((r.out[1:].double() - r.out[0].double()).abs().max()) <= 2.0 ** -7 * float(r.out.double().abs().max())


def test_refusals_of_the_binding():
    torch = torch_cuda()
    a = plain_call()

    def refused(**kw):
        with pytest.raises(ts.TopSelectError):
            ts.ts_cache_attend(**{**a, **kw})
    refused(q=a["q"].float())
    refused(q=a["q"][0])
    refused(q=a["q"].transpose(1, 2))
    refused(k_pages=a["k_pages"][:, :, :8])
    refused(k_pages=a["k_pages"].cpu())
    refused(table=a["table"].long())
    refused(table=a["table"][:2])
    refused(table=a["table"].t())
    refused(lengths=a["lengths"].long())
    refused(lengths=None)
    refused(weights_dtype=torch.int32)
    refused(weights_slots=-1)
    refused(scale=-1.0)
    refused(window=-1)
    refused(out=torch.empty(3, 6, 64, device="cuda"))
    refused(out=torch.empty(1, 6, 64, dtype=a["q"].dtype, device="cuda").expand(3, 6, 64))
    refused(q=torch.empty(3, 5, 64, dtype=a["q"].dtype, device="cuda"))
    assert not host(ts.ts_cache_attend(**a).status).any()


@pytest.mark.parametrize("n", [511, 512, 513, 1000, 1024, 1025])
def test_rows_of_one_workgroup_and_of_several(n):
    rng = np.random.default_rng(n)
    check(lengths=np.r_[n, rng.integers(0, n + 1, 3)], wtype="float32", hk=1, hq=5)
    check(lengths=np.r_[n, rng.integers(0, n + 1, 130)], hk=2, hq=2, dim=16, dtype="float16")      # rows enough for the chip
    check(lengths=[5 * n, n], window=n, hk=1, hq=2, dtype="float32")


@pytest.mark.parametrize("seed", range(12))
def test_random_batches(seed):
    rng = np.random.default_rng(1000 + seed)
    hk, group = int(rng.choice([1, 2, 3])), int(rng.choice([1, 2, 5, 16, 20]))
    lengths = np.exp(rng.uniform(0, np.log(3000), int(rng.integers(1, 12)))).astype(int)
    lengths[rng.random(len(lengths)) < 0.1] = 0
    check(lengths=lengths, hk=hk, hq=hk * group, dim=int(rng.choice([5, 16, 64, 100, 128, 250])), slots=int(rng.choice([1, 7, 16, 48, 500])),
          dtype=TYPES[seed % 3], window=int(rng.choice([0, 0, 40, 700])), wtype=[None, "float32", "bfloat16", "float16"][seed % 4],
          seed=seed, slots_first=bool(seed & 1))


@pytest.mark.parametrize("n", [40, 600])
def test_more_rows_than_65535(n):
    """9000 times the same sequence of 8 heads: every one has the first one's bits, or the next ones' of another share."""
    torch = torch_cuda()
    a = plain_call(3, batch=1, n=n)
    k, v = (a[x][:, :1].expand(-1, 8, -1, -1).contiguous() for x in ("k_pages", "v_pages"))
    q = a["q"][:, :1].expand(9000, 8, 64).contiguous()
    lengths = torch.full((9000,), n - 1, dtype=torch.int32, device="cuda")
    r = ts.ts_cache_attend(q, k, v, a["table"].expand(9000, -1).contiguous(), lengths)
    want = paged.attend_row(host(q[:1].double())[0], host(k.double()), host(v.double()), a["table"][0].tolist(), n - 1, 0.125, 0, 0)
    compare(want, host(r.out[0].double()), host(r.lse[0].double()), None, 0.125, "bfloat16", None, 1, "first")
    # shares end at other positions of the row, which changes the sums' order: within a half step of each other, and a few u
    assert float((r.out.double() - r.out[0, 0].double()).abs().max()) <= 2.0 ** -7 * float(r.out[0, 0].double().abs().max())
    assert float((r.lse.double() - r.lse[0, 0].double()).abs().max()) < 1e-5 and not bool(r.status.any())


def test_many_tiny_sequences_beside_long_ones():
    """Rows of one tile each fall to a few waves; one row spans many workgroups."""
    lengths = np.r_[np.arange(1, 60), 30000, np.ones(40, int), 12000]
    check(lengths=lengths, hk=1, hq=3, dim=64, slots=16, dtype="bfloat16", wtype="float32")


def weights_of_a_spoilt_score(route, dtype, wtype, value, window):
    """Sequence 0 attends a key that makes one head's score NaN or +inf; sequence 1's page number is bad; 2 is sound, 3 empty.
    Of 0's spoilt heads every attended weight is NaN (so is the sum), every other slot 0: only rejected sequences have NaN there."""
    torch = torch_cuda()
    # one launch; several workgroups' stretches with rows that one of them finishes; a row that many of them share
    n, room, batch = {"whole": (90, 128, 4), "finished": (90, 2000, 4000), "joined": (9000, 9100, 4)}[route]
    gen = torch.Generator(device="cuda").manual_seed(n)
    t, slots, dim = getattr(torch, dtype), 16, 32
    width, held = -(-room // slots), -(-n // slots)
    k, v = (torch.randn((4 * held, 2, slots, dim), generator=gen, device="cuda").to(t) for _ in range(2))
    table = torch.full((batch, width), -1, dtype=torch.int32, device="cuda")
    table[:4, :held] = torch.arange(4 * held, dtype=torch.int32, device="cuda").view(4, held)
    table[4:, :held] = table[2, :held]
    q = torch.randn((batch, 6, dim), generator=gen, device="cuda").to(t)
    q[:, 3:, 0] = 1.0
    lengths = torch.full((batch,), n, dtype=torch.int32, device="cuda")
    lengths[3] = 0
    at = n - 20                                                   # inside every window
    k[table[0, at // slots].long(), 1, at % slots, 0] = value     # of heads 3, 4 and 5
    table[1, (n - 1) // slots] = 1 << 30
    banner(f"attend: weights of a spoilt score {route} {dtype} {wtype} {value} window={window}")
    r = ts.ts_cache_attend(q, k, v, table, lengths, window=window, weights_slots=n + 7, weights_dtype=getattr(torch, wtype))
    status, w = host(r.status), host(r.weights[:4].double())
    assert status[:4].tolist() == [0, ts.TS_ROW_BAD_PAGE, 0, 0] and not status[4:].any()
    lo = max(0, n - window) if window else 0
    attended = np.zeros(n + 7, bool)
    attended[lo:n] = True
    for h in range(6):
        if h >= 3:
            assert np.isnan(w[0, h, attended]).all() and np.isnan(host(r.out[0, h].double())).all() and np.isnan(float(r.lse[0, h]))
        else:
            assert (w[0, h, attended] > 0).any() and np.isfinite(w[0, h]).all()
        for b in (0, 2):
            assert (w[b, h, ~attended] == 0).all(), f"head {h} of sequence {b}: weights outside its positions"
        assert np.isfinite(w[2, h]).all() and not w[3, h].any() and np.isnan(w[1, h]).all()


@pytest.mark.parametrize("route", ["whole", "finished", "joined"])
@pytest.mark.parametrize("dtype,wtype", [("bfloat16", "bfloat16"), ("float32", "float32"), ("float16", "float32")])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_weights_outside_the_positions_of_a_spoilt_score(route, dtype, wtype, value):
    for window in (0, 37):
        weights_of_a_spoilt_score(route, dtype, wtype, value, window)


@pytest.mark.parametrize("window", [(1 << 31) - 1, 1 << 31, (1 << 32) + 5, 1 << 62])
def test_windows_past_any_length(window):
    a = plain_call(4)
    assert equal(ts.ts_cache_attend(**a, window=window), ts.ts_cache_attend(**a))
    with pytest.raises(ts.TopSelectError):
        ts.ts_cache_attend(**a, window=-window)


def test_output_between_the_queries_of_one_buffer():
    """[batch, 2, heads, dim]: queries and outputs by turns are accepted and leave each other alone; shifted into them they are refused."""
    torch = torch_cuda()
    a = plain_call(8)
    want = ts.ts_cache_attend(**a)
    buf = torch.zeros(3, 2, 6, 64, dtype=a["q"].dtype, device="cuda")
    buf[:, 0] = a["q"]
    r = ts.ts_cache_attend(**{**a, "q": buf[:, 0]}, out=buf[:, 1])
    assert equal(r, want) and torch.equal(buf[:, 0], a["q"]) and torch.equal(buf[:, 1], want.out)
    flat = torch.zeros(3 * 6 * 64 + 64, dtype=a["q"].dtype, device="cuda")
    q, out = flat[:-64].view(3, 6, 64), flat[64:].view(3, 6, 64)
    with pytest.raises(ts.TopSelectError, match="overlaps"):
        ts.ts_cache_attend(**{**a, "q": q}, out=out)
    with pytest.raises(ts.TopSelectError):
        ts.ts_cache_attend(**{**a, "q": q}, out=q)
