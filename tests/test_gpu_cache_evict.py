"""GPU tests of ts_cache_evict against the oracle: which slots stay, where they go, their weights (equal in every
bit: a binary64 sum in the oracle's order, rounded once) and the moved caches."""
import math

import numpy as np
import pytest

import oracle
import top_select_gumbel_amd as ts
from gpu_helpers import banner, host, torch_cuda

pytestmark = pytest.mark.gpu


def gpu(a, dtype=None):
    torch = torch_cuda()
    t = torch.from_numpy(np.ascontiguousarray(a))
    return (t if dtype is None else t.to(getattr(torch, dtype))).cuda()


def caches(batch, heads, slots, dim, dtype, seed, slots_first=False, wide=0):
    """A cache of random bit patterns; `slots_first`: [batch, slots, heads, dim] in memory; `wide`: unused elements a slot."""
    torch = torch_cuda()
    size = torch.empty(0, dtype=getattr(torch, dtype)).element_size()
    shape = (batch, slots, heads, dim + wide) if slots_first else (batch, heads, slots, dim + wide)
    raw = np.random.default_rng(seed).integers(0, 120, shape[:3] + (shape[3] * size,), dtype=np.uint8)
    t = torch.from_numpy(raw).cuda().view(getattr(torch, dtype))
    return (t.transpose(1, 2) if slots_first else t)[..., :dim]


def bits(t):
    return host(t.contiguous().view(torch_cuda().uint8))


def check(batch, heads, slots, keep, n_w=2, wtype="float32", dim=16, ctype="bfloat16", v_dim=None, lengths=None, keeps=None, sinks=0,
          recent=0, ties=0, seed=0, permuted=True, in_place=False, slots_first=False, wide=0, score=None, weights=None, pad=0):
    torch = torch_cuda()
    banner(f"evict b={batch} h={heads} slots={slots} keep={keep} n_w={n_w} {wtype} {ctype} dim={dim} sinks={sinks} recent={recent}")
    rng = np.random.default_rng(seed)
    rows = batch * heads
    if score is None:
        score = rng.integers(0, ties, (rows, slots)).astype(np.float32) if ties else rng.standard_normal((rows, slots)).astype(np.float32)
    if weights is None:
        weights = rng.integers(0, 2, (rows, n_w, slots)) if ties else rng.random((rows, n_w, slots))
    w = gpu(weights.astype(np.float32), wtype) if n_w else None
    lengths = np.full(rows, slots, np.int32) if lengths is None else np.asarray(lengths, np.int32)
    keeps = np.full(rows, keep, np.int32) if keeps is None else np.asarray(keeps, np.int32)
    position = np.stack([rng.permutation(slots) if permuted else np.arange(slots) for _ in range(rows)]).astype(np.int32)

    def padded(a):   # rows further apart than they are long
        t = gpu(np.pad(a, ((0, 0), (0, pad))))
        return t[:, :slots]
    k = caches(batch, heads, slots, dim, ctype, seed + 1, slots_first, wide)
    v = caches(batch, heads, slots, v_dim or dim, ctype, seed + 2, slots_first, wide)
    whole = [t._base if t._base is not None else t for t in (k, v)]
    before = [bits(t) for t in (k, v)] + [bits(t) for t in whole]
    args = (padded(score), padded(position), gpu(lengths), gpu(keeps))
    r = ts.ts_cache_evict(*args, keep, weights=w, k_cache=k, v_cache=v, sinks=sinks, recent=recent, in_place=in_place)
    torch.cuda.synchronize()
    src, length, sc, pos, st = (host(t) for t in r)
    after = [bits(t) for t in (k, v)]
    ws = np.zeros((rows, 0, slots)) if w is None else w.double().cpu().numpy()
    for i in range(rows):
        n = int(np.clip(lengths[i], 0, slots))
        o = oracle.cache_evict_row(score[i], ws[i], position[i], n, int(keeps[i]), keep, sinks, recent)
        where = f"row {i} n={n} keep={keeps[i]}"
        assert st[i] == o.status and length[i] == o.length, where
        b, h = divmod(i, heads)
        if o.status:
            assert (src[i] == -1).all(), where
            if in_place:
                assert np.array_equal(sc[i], score[i], equal_nan=True) and np.array_equal(pos[i], position[i]), where
            else:
                assert np.isnan(sc[i]).all() and (pos[i] == -1).all(), where
            for was, now in zip(before, after):
                assert np.array_equal(was[b, h], now[b, h]), where
            continue
        m = o.length
        assert src[i, :m].tolist() == o.source and (src[i, m:] == -1).all(), where
        assert np.array_equal(sc[i, :m].view(np.uint32), o.score.view(np.uint32)), where
        assert np.array_equal(pos[i, :m], o.position), where
        assert not sc[i, m:keep].any() and (pos[i, m:keep] == -1).all(), where
        if in_place:        # nothing past the widest row is written
            assert np.array_equal(sc[i, keep:], score[i, keep:], equal_nan=True) and np.array_equal(pos[i, keep:], position[i, keep:])
        for was, now in zip(before, after):
            assert np.array_equal(now[b, h, :m], was[b, h][np.array(o.source, int)]), where
            assert np.array_equal(now[b, h, m:], was[b, h, m:]), where      # slots behind the cut stay as they were
    if wide:                # the unused elements of a slot
        for t, was, dim_ in ((whole[0], before[2], dim), (whole[1], before[3], v_dim or dim)):
            size = t.element_size()
            assert np.array_equal(bits(t)[..., dim_ * size:], was[..., dim_ * size:])
    return r


@pytest.mark.parametrize("slots,keep", [(1, 1), (2, 1), (3, 2), (63, 40), (64, 64), (65, 1), (200, 199), (1025, 1024), (1500, 300), (5000, 2500)])
@pytest.mark.parametrize("wtype", ["float32", "bfloat16", "float16"])
def test_sizes(slots, keep, wtype):
    check(2, 3, slots, keep, wtype=wtype, seed=slots)
    check(1, 2, slots, keep, wtype=wtype, seed=slots, sinks=2, recent=5, permuted=False, pad=3)


def test_ragged_lengths_and_keeps():
    n = [0, 1, 2, 300, 299, 77, 150, 151, -4, 999]
    for in_place in (False, True):
        check(5, 2, 300, 150, lengths=n, keeps=[150, 1, 1, 150, 149, 150, 150, 150, 3, 1], sinks=1, recent=3, seed=3, in_place=in_place)


@pytest.mark.parametrize("slots", [50, 1300, 3000])
def test_ties_go_to_the_lowest_slot(slots):
    check(2, 2, slots, slots // 2, ties=3, seed=slots)
    check(2, 2, slots, slots // 3, ties=2, n_w=0, seed=slots, sinks=3, recent=9)
    zeros = np.zeros((4, slots), np.float32)
    zeros[1:, ::2] = -0.0                              # -0 is 0
    check(2, 2, slots, slots // 2, n_w=0, score=zeros, seed=1)


@pytest.mark.parametrize("sinks,recent", [(0, 0), (4, 0), (0, 16), (4, 64), (300, 0), (0, 300), (2 ** 31 - 1, 0), (0, 2 ** 31 - 1), (90, 90)])
def test_protected_positions(sinks, recent):
    # from none to more than fit: among protected ones the weight decides
    check(2, 2, 300, 100, sinks=sinks, recent=recent, seed=sinks % 97 + recent % 89)
    check(1, 2, 300, 100, sinks=sinks, recent=recent, ties=2, n_w=1, seed=7)


@pytest.mark.parametrize("ctype,dim,v_dim", [("bfloat16", 128, None), ("float16", 33, 80), ("float32", 5, 1), ("uint8", 7, 16), ("uint8", 1, 3),
                                             ("bfloat16", 4, 512), ("float32", 96, 2)])
@pytest.mark.parametrize("layout", ["heads", "slots", "wide"])
def test_cache_types_and_layouts(ctype, dim, v_dim, layout):
    check(2, 3, 130, 61, dim=dim, ctype=ctype, v_dim=v_dim, slots_first=layout == "slots", wide=3 if layout == "wide" else 0, seed=dim)


@pytest.mark.parametrize("dim,v_dim", [(15, 16), (16, 17), (17, 15), (31, 33), (257, 31), (4099, 16)])
@pytest.mark.parametrize("layout", ["heads", "slots", "wide"])
def test_slots_of_any_size_and_address(dim, v_dim, layout):
    """Bytes, so that slots start anywhere and end inside a copy's unit."""
    for slots, keep in ((130, 61), (2500, 1200), (8300, 90)):
        if dim * slots < 1 << 21:
            check(1, 3, slots, keep, dim=dim, ctype="uint8", v_dim=v_dim, slots_first=layout == "slots",
                  wide=3 if layout == "wide" else 0, seed=dim)


@pytest.mark.parametrize("slots", [40, 2048, 2049, 9000])
def test_keep_may_exceed_the_slots(slots):
    check(2, 2, slots, slots + 300, lengths=[slots, 3, 0, slots - 1], dim=4, seed=slots)
    check(2, 2, slots, slots + 300, lengths=[slots, 3, 0, slots - 1], keeps=[5, 2, 1, slots // 2], dim=4, seed=slots)


def test_many_short_rows():
    check(60, 10, 90, 41, n_w=1, dim=6, sinks=1, recent=4, seed=5)


@pytest.mark.parametrize("slots", [300, 9000])
def test_shared_weights_and_one_tensor_as_both_caches(slots):
    """Weights broadcast over rows and over the weight rows, and keys that are their own values."""
    torch = torch_cuda()
    rng = np.random.default_rng(3)
    score = gpu(rng.random((4, slots)).astype(np.float32))
    position = gpu(np.tile(np.arange(slots, dtype=np.int32), (4, 1)))
    n, keep = gpu(np.full(4, slots, np.int32)), gpu(np.full(4, slots // 3, np.int32))
    one = gpu(rng.random((1, 1, slots)).astype(np.float32))
    k = caches(2, 2, slots, 8, "bfloat16", 3)
    k2 = k.clone()
    a = ts.ts_cache_evict(score, position, n, keep, slots // 3, weights=one.expand(4, 3, slots).contiguous(), k_cache=k)
    b = ts.ts_cache_evict(score, position, n, keep, slots // 3, weights=one.expand(4, 3, slots), k_cache=k2, v_cache=k2)
    assert all(torch.equal(x, y) for x, y in zip(a, b)) and torch.equal(k, k2)
    c = ts.ts_cache_evict(score, position, n, keep, slots // 3, weights=one.expand(4, 3, slots)[:, :0])
    d = ts.ts_cache_evict(score, position, n, keep, slots // 3)
    assert all(torch.equal(x, y) for x, y in zip(c, d))


def test_one_cache_or_none():
    torch = torch_cuda()
    rng = np.random.default_rng(2)
    score, position = gpu(rng.random((4, 50)).astype(np.float32)), gpu(np.tile(np.arange(50, dtype=np.int32), (4, 1)))
    lengths, keep = gpu(np.full(4, 50, np.int32)), gpu(np.full(4, 20, np.int32))
    k = caches(2, 2, 50, 8, "float32", 1)
    a = ts.ts_cache_evict(score, position, lengths, keep, 20)
    b = ts.ts_cache_evict(score, position, lengths, keep, 20, v_cache=k)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    want = host(k)
    c = ts.ts_cache_evict(score, position, lengths, keep, 20, k_cache=k)      # same slots again: nothing new moves
    assert all(torch.equal(x, y) for x, y in zip(a, c)) and np.array_equal(host(k), want)


@pytest.mark.parametrize("in_place", [False, True])
def test_rejected_rows_stay_as_they_are(in_place):
    rng = np.random.default_rng(4)
    score = rng.standard_normal((8, 90)).astype(np.float32)
    w = rng.random((8, 2, 90)).astype(np.float32)
    score[0, 5], score[1, 80], w[2, 1, 3], w[3, 0, 7] = math.nan, math.inf, math.nan, -math.inf
    score[4, 70:], w[5, :, 70:] = math.nan, math.inf       # behind their rows' ends
    n = [90, 90, 90, 90, 70, 70, 90, 90]
    check(4, 2, 90, 40, score=score, weights=w, lengths=n, keeps=[40] * 6 + [0, 41], in_place=in_place)


def test_infinite_sum_is_rejected():
    score = np.full((2, 8), 3e38, np.float32)
    check(1, 2, 8, 4, score=score, weights=np.full((2, 1, 8), 3e38), n_w=1)


def test_sums_are_wide():
    # 4096 + 1000 * 2^-13: fp32 steps of 2^-11 would lose every addend
    score = np.full((1, 4), 4096.0, np.float32)
    w = np.full((1, 1000, 4), 2.0 ** -13)
    w[0, :, 1] = 0
    r = check(1, 1, 4, 3, n_w=1000, score=score, weights=w)
    assert host(r.score)[0, 0] == np.float32(4096 + 1000 * 2.0 ** -13)


def test_negative_positions_and_weights():
    torch = torch_cuda()
    score = gpu(-np.arange(1, 9, dtype=np.float32)[None])
    position = gpu(np.array([[-2 ** 31, -5, 3, 2 ** 31 - 1, 7, 8, 9, 10]], np.int32))
    r = ts.ts_cache_evict(score, position, gpu(np.array([8], np.int32)), gpu(np.array([3], np.int32)), 3, recent=1)
    assert host(r.source).tolist() == [[0, 1, 3]]
    r = ts.ts_cache_evict(score, position, gpu(np.array([8], np.int32)), gpu(np.array([3], np.int32)), 3, sinks=1)
    assert host(r.source).tolist() == [[0, 1, 2]]
    assert host(r.position).tolist() == [[-2 ** 31, -5, 3]]


@pytest.mark.parametrize("slots,keep,batch", [(40000, 5000, 2), (70001, 69990, 1), (33000, 3, 3)])
def test_long_rows(slots, keep, batch):
    check(batch, 1, slots, keep, n_w=1, wtype="bfloat16", dim=8, sinks=4, recent=32, seed=slots)
    check(batch, 1, slots, keep, n_w=1, wtype="bfloat16", dim=8, ties=2, seed=slots)


@pytest.mark.parametrize("in_place", [False, True])
def test_long_ragged_and_rejected_rows(in_place):
    slots = 9000
    rng = np.random.default_rng(11)
    score = rng.standard_normal((10, slots)).astype(np.float32)
    score[4, 8000] = math.nan
    score[5, 8500:] = math.nan                          # behind its row's end
    n = [0, 1, 9000, 8999, 9000, 8500, 1024, 1025, -3, 12000]
    check(5, 2, slots, 4000, score=score, lengths=n, keeps=[4000, 1, 3999, 4000, 4000, 1, 1024, 1024, 4000, 0], sinks=3, recent=700,
          dim=4, in_place=in_place, seed=11)


@pytest.mark.parametrize("slots", [8192, 8193, 9216, 20000])
@pytest.mark.parametrize("sinks,recent", [(0, 0), (5000, 0), (10, 6000), (2 ** 31 - 1, 0)])
def test_long_protected_positions(slots, sinks, recent):
    check(1, 2, slots, 5000, sinks=sinks, recent=recent, dim=2, seed=slots)
    check(1, 2, slots, slots, sinks=sinks, recent=recent, dim=2, seed=slots)
    check(1, 1, slots, 5000, sinks=sinks, recent=recent, dim=2, ties=2, n_w=1, seed=slots)


@pytest.mark.parametrize("slots,keep", [(8193, 8000), (16384, 900), (16385, 16000), (12000, 12000)])
def test_many_rows_of_middle_length(slots, keep):
    # 64 rows and more are held in registers up to 16384 slots
    check(16, 4, slots, keep, n_w=1, wtype="bfloat16", dim=2, ctype="uint8", sinks=4, recent=50, seed=slots,
          lengths=[slots - (i * 977) % slots for i in range(64)])
    check(16, 4, slots, keep, n_w=1, dim=2, ctype="uint8", ties=2, seed=slots)


@pytest.mark.parametrize("slots", [3000, 20000])
def test_outliers_crowd_the_other_weights_together(slots):
    # one huge weight stretches the row's range, so that all others share a few of the first bins
    rng = np.random.default_rng(slots)
    score = (1 + rng.random((3, slots))).astype(np.float32)
    score[0, 7], score[1, 7], score[1, 9] = 1e30, 1e30, -1e30
    score[2] = np.round(score[2] * 64) / 64             # and many ties besides
    score[2, 7] = 1e30
    check(3, 1, slots, slots // 3, n_w=0, score=score, dim=2, seed=1)


def test_steps_in_a_row_against_the_oracle():
    """A cache at its budget over many steps: append, add the step's weights, drop one; in place throughout."""
    torch = torch_cuda()
    rng = np.random.default_rng(8)
    heads, budget, dim = 3, 40, 12
    slots = budget + 1
    score, position = torch.zeros(heads, slots, device="cuda"), torch.full((heads, slots), -1, dtype=torch.int32, device="cuda")
    lengths, keep = torch.zeros(heads, dtype=torch.int32, device="cuda"), torch.full((heads,), budget, dtype=torch.int32, device="cuda")
    k = torch.zeros(1, heads, slots, dim, device="cuda")
    held = [dict() for _ in range(heads)]               # oracle: slot -> (weight, position)
    for step in range(120):
        at = lengths.long()[:, None]
        score.scatter_(1, at, 0.0)
        position.scatter_(1, at, step)
        k[0].scatter_(1, at[:, :, None].expand(-1, -1, dim), float(step))
        lengths += 1
        w = rng.random((heads, 2, slots)).astype(np.float32)
        r = ts.ts_cache_evict(score, position, lengths, keep, budget, weights=gpu(w), k_cache=k, sinks=2, recent=8, in_place=True)
        torch.cuda.synchronize()
        for h in range(heads):
            held[h][len(held[h])] = (0.0, step)
            n = len(held[h])
            o = oracle.cache_evict_row([held[h][j][0] for j in range(n)], w[h], [held[h][j][1] for j in range(n)], n, budget, budget, 2, 8)
            held[h] = {j: (float(o.score[j]), int(o.position[j])) for j in range(o.length)}
            assert int(lengths[h]) == o.length
            assert host(position[h, :o.length]).tolist() == o.position.tolist()
            assert np.array_equal(host(score[h, :o.length]), o.score)
            assert np.array_equal(host(k[0, h, :o.length, 0]), o.position.astype(np.float32))   # keys move with their positions


def test_streams_and_graphs():
    torch = torch_cuda()
    rng = np.random.default_rng(6)
    def inputs(seed):
        g = np.random.default_rng(seed)
        return (gpu(g.random((8, 700)).astype(np.float32)), gpu(np.tile(np.arange(700, dtype=np.int32), (8, 1))),
                gpu(g.integers(1, 701, 8).astype(np.int32)), gpu(np.full(8, 200, np.int32)))
    cases = [inputs(s) for s in (1, 2)]
    ks = [caches(2, 4, 700, 32, "bfloat16", s) for s in (5, 6)]
    want = []
    for c, k in zip(cases, ks):
        k2 = k.clone()
        want.append((ts.ts_cache_evict(*c, 200, k_cache=k2, sinks=1, recent=4), k2))
    torch.cuda.synchronize()
    streams, graphs = [torch.cuda.Stream(), torch.cuda.Stream()], []
    for c, k in zip(cases, ks):
        work = k.clone()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = ts.ts_cache_evict(*c, 200, k_cache=work, sinks=1, recent=4)
        graphs.append((g, out, work))
    for _ in range(3):
        for (g, _, work), k in zip(graphs, ks):
            work.copy_(k)
        torch.cuda.synchronize()
        for (g, _, _), s in zip(graphs, streams):        # both at once
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        torch.ones(500, device="cuda").sum().item()
        for (_, out, work), (w, wk) in zip(graphs, want):
            assert all(torch.equal(a, b) for a, b in zip(out, w)) and torch.equal(work, wk)


def test_empty_batch_and_refusals():
    torch = torch_cuda()
    score, position = torch.zeros(4, 20, device="cuda"), torch.zeros(4, 20, dtype=torch.int32, device="cuda")
    n = torch.full((4,), 20, dtype=torch.int32, device="cuda")
    r = ts.ts_cache_evict(score[:0], position[:0], n[:0], n[:0], 5)
    assert r.source.shape == (0, 5)
    k = torch.zeros(2, 2, 20, 8, device="cuda")
    shared = torch.zeros(2, 1, 20, 8, device="cuda").expand(2, 2, 20, 8)
    good = dict(score=score, position=position, lengths=n, keep=n, keep_max=5)
    for bad in (dict(score=score.double()), dict(score=score.t()), dict(position=position.long()), dict(position=position[:, :19]),
                dict(lengths=n[:3]), dict(lengths=None), dict(keep=n.long()), dict(keep_max=0), dict(keep_max=21, in_place=True),
                dict(weights=torch.zeros(4, 20, device="cuda")), dict(weights=torch.zeros(4, 2, 19, device="cuda")),
                dict(weights=torch.zeros(4, 2, 20, device="cuda").double()), dict(weights=torch.zeros(4, 20, 2, device="cuda").transpose(1, 2)),
                dict(k_cache=k[:1]), dict(k_cache=k[:, :, :19]), dict(k_cache=k.transpose(2, 3)), dict(k_cache=shared), dict(k_cache=k[..., ::2]),
                dict(k_cache=k, v_cache=k.view(1, 4, 20, 8)), dict(k_cache=k.cpu()), dict(sinks=-1), dict(recent=-1)):
        with pytest.raises(ts.TopSelectError):
            ts.ts_cache_evict(**{**good, **bad})
    assert not k.any()
