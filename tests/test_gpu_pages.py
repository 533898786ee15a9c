"""GPU tests of ts_cache_append, ts_pages_fork, ts_pages_compact and ts_pages_copy against the oracle: whole numbers and bytes,
equal in every bit."""
import numpy as np
import pytest

from oracle import paged
import top_select_gumbel_amd as ts
from gpu_helpers import banner, host, torch_cuda

pytestmark = pytest.mark.gpu


def gpu(a):
    return torch_cuda().from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def pool_of(pages, shape, dtype, seed, gap=0):
    """Random bit patterns; `gap`: unused elements between pages."""
    torch = torch_cuda()
    t = getattr(torch, dtype)
    size = torch.empty(0, dtype=t).element_size()
    n = int(np.prod(shape)) + gap
    raw = np.random.default_rng(seed).integers(0, 256, (pages, n * size), dtype=np.uint8)
    flat = torch.from_numpy(raw).cuda().view(t)
    return flat[:, : n - gap].view(pages, *shape) if not gap else flat.as_strided((pages, n - gap), (n, 1))


def same(a, b, what):
    """Equality without the two arrays' print."""
    equal = a.shape == b.shape and np.array_equal(a, b)
    assert equal, f"{what} differs at {np.argwhere(a != b)[:5].tolist() if a.shape == b.shape else (a.shape, b.shape)}"


def raw(t):
    torch = torch_cuda()
    return host((t._base if t._base is not None else t).contiguous().view(torch.uint8)).copy()


def moved(before, pool, moves):
    """The bytes that the pool's storage should hold."""
    torch = torch_cuda()
    want = torch.from_numpy(before.copy())
    whole = want.view(pool.shape[0], -1)
    page = pool[0].numel() * pool.element_size()
    src = whole.clone()
    for a, b in moves:
        whole[b, :page] = src[a, :page]
    return want.numpy()


# ---------------------------------------------------------------- append
def check_append(lengths, new, slots=16, heads=2, dim=16, dtype="bfloat16", spare=0, extra_pages=3, edit=None, seed=0, slots_first=False,
                 strided=False, pages_too=True):
    torch = torch_cuda()
    lengths, new = np.asarray(lengths, np.int32), np.asarray(new, np.int32)
    banner(f"append n={lengths[:5].tolist()} new={new[:5].tolist()} slots={slots} heads={heads} dim={dim} {dtype}")
    b, width = len(lengths), max(1, -(-int(max(lengths, default=1)) // slots))
    pages = b * width + extra_pages
    rng = np.random.default_rng(seed)
    table = rng.permutation(pages)[: b * width].reshape(b, width).astype(np.int32)
    offsets = np.r_[0, np.cumsum(new)].astype(np.int32)
    tokens = int(offsets[-1]) + spare
    if edit is not None:
        edit(table, lengths, offsets)
    shape = (slots, heads, dim) if slots_first else (heads, slots, dim)
    k, v = (pool_of(pages, shape, dtype, seed + i) for i in (1, 2))
    kv = [x.transpose(1, 2) if slots_first else x for x in (k, v)]
    fresh = [pool_of(max(tokens, 1), (heads, 2 * dim if strided else dim), dtype, seed + i)[:tokens, :, :dim] for i in (3, 4)]
    want = [host(x.contiguous().view(torch.uint8)).reshape(pages, heads, slots, -1).copy() for x in kv]
    new_bytes = [host(x.contiguous().view(torch.uint8)).reshape(tokens, heads, dim * x.element_size()) for x in fresh]
    st = ts.ts_cache_append(fresh[0], fresh[1], gpu(offsets), kv[0], kv[1], gpu(table), gpu(lengths))
    torch.cuda.synchronize()
    moves, status = paged.append(lengths.tolist(), offsets.tolist(), table.tolist(), slots, pages, tokens)
    for t, p, s in moves:
        for w, x in zip(want, new_bytes):
            w[p, :, s] = x[t]
    assert host(st).tolist() == status
    for got, w in zip(kv, want):
        if pages_too:
            same(host(got.contiguous().view(torch.uint8)).reshape(w.shape), w, "cache")


@pytest.mark.parametrize("dtype,dim", [("bfloat16", 128), ("float32", 33), ("float16", 1), ("uint8", 7), ("float32", 1024), ("bfloat16", 33)])
def test_append_types_and_sizes(dtype, dim):
    check_append([5, 17, 16, 1, 40], [1, 1, 1, 1, 1], dtype=dtype, dim=dim)
    check_append([5, 17, 16, 1, 40], [5, 3, 0, 1, 40], dtype=dtype, dim=dim, slots=7)


@pytest.mark.parametrize("slots", [1, 5, 16, 64])
@pytest.mark.parametrize("slots_first,strided", [(False, False), (True, True)])
def test_append_layouts(slots, slots_first, strided):
    check_append([100, 3, 64, 0, 77], [100, 2, 0, 0, 1], slots=slots, slots_first=slots_first, strided=strided, heads=3)


def test_append_many_and_none():
    rng = np.random.default_rng(1)
    n = rng.integers(0, 60, 500)
    check_append(n, np.minimum(n, rng.integers(0, 9, 500)), dim=8)
    check_append([3, 4], [0, 0])
    check_append([3, 4], [2, 4], spare=6)          # tokens behind the last sequence's go nowhere


def test_append_statuses():
    def edit(table, lengths, offsets):
        table[1, 0], table[2, 1] = -1, 1 << 30
        lengths[3], lengths[4] = 2, 1000
    check_append([20, 20, 20, 20, 20, 20], [4, 20, 8, 3, 1, 2], edit=edit)

    def torn(table, lengths, offsets):             # offsets that go down, or past the tokens
        offsets[2], offsets[5] = 1, 99
    check_append([20, 20, 20, 20, 20, 20], [4, 2, 8, 3, 1, 2], edit=torn, pages_too=False)   # which of two takes a token is left open

    def negative(table, lengths, offsets):
        offsets[0], lengths[1] = -3, -5
    check_append([20, 20, 20], [4, 2, 8], edit=negative)


# ---------------------------------------------------------------- fork
def check_fork(table, lengths, refs, parent, new, slots, width=None, pools=2, page=(2, 16, 8), dtype="bfloat16", in_place=False, seed=0,
               gap=0, spread=0):
    torch = torch_cuda()
    table = np.asarray(table, np.int32)
    width = table.shape[1] if width is None else width
    banner(f"fork seqs={len(lengths)} children={len(parent)} pages={len(refs)} slots={slots} width={table.shape[1]}->{width} pools={pools}")
    p = [pool_of(len(refs), page if i % 3 else (3,) + tuple(page[1:]), dtype, seed + i, gap) for i in range(pools)]
    before = [raw(x) for x in p]
    t = gpu(table)
    if spread:      # rows further apart than they are long
        t = torch.nn.functional.pad(t, (0, spread), value=1 << 29)[:, : table.shape[1]]
    r0 = gpu(refs)
    r = ts.ts_pages_fork(t, gpu(lengths), r0, gpu(parent), slots, n_new=None if new is None else gpu(new), pools=p, width=width,
                         in_place=in_place)
    torch.cuda.synchronize()
    o = paged.fork(table.tolist(), list(lengths), refs, list(parent), [0] * len(parent) if new is None else list(new), slots, width)
    assert host(r.status).tolist() == o.status
    assert host(r.lengths).tolist() == o.lengths
    assert host(r.table).tolist() == o.table
    assert host(r.refs).tolist() == o.refs
    if in_place:
        assert r.refs.data_ptr() == r0.data_ptr()
    else:
        assert host(r0).tolist() == list(refs)
    for x, b in zip(p, before):
        same(raw(x).ravel(), moved(b, x, o.copies).ravel(), "pool")
    return r


def sequences(rng, seqs, pages, slots, width, share=0.3, fill=0.6):
    """Tables after some life: pages in no order, some of them shared, counts to match."""
    order = rng.permutation(pages).tolist()
    table, lengths = [], []
    for s in range(seqs):
        room = min(width * slots, int(fill * pages / seqs * slots * 2))
        n = int(rng.integers(0, max(room, 1) + 1))
        row = []
        if table and rng.random() < share:
            donor = int(rng.integers(0, len(table)))
            row = table[donor][: min(lengths[donor] // slots, n // slots)]
        need = -(-n // slots) - len(row)
        if need > len(order):
            n, row, need = 0, [], 0
        row = list(row) + [order.pop() for _ in range(need)]
        table.append(row + [int(rng.integers(-5, pages + 5)) for _ in range(width - len(row))])
        lengths.append(n)
    refs = [0] * pages
    for row, n in zip(table, lengths):
        for p in row[: -(-n // slots)]:
            refs[p] += 1
    return table, lengths, refs


@pytest.mark.parametrize("seed", range(24))
def test_fork_random(seed):
    rng = np.random.default_rng(seed)
    pages, slots, seqs = int(rng.integers(3, 300)), int(rng.choice([1, 3, 16, 50])), int(rng.integers(1, 30))
    width = int(rng.integers(1, 40))
    table, lengths, refs = sequences(rng, seqs, pages, slots, width)
    n = int(rng.integers(1, 40))
    parent = rng.integers(-1, seqs, n) if seed % 3 else np.where(np.arange(n) < seqs, np.arange(n), -1)
    new = rng.integers(0, [2, 2 * slots, 10 * slots][seed % 3], n)
    if seed % 4 == 3:
        new[rng.integers(0, n)] = [-1, 1 << 30, (1 << 31) - 1][seed % 3]
        parent[rng.integers(0, n)] = [-2, seqs, 1 << 30][seed % 3]
    check_fork(table, lengths, refs, parent, new, slots, width=width + int(rng.integers(-1, 3)) if seed % 2 else None,
               in_place=bool(seed % 2), seed=seed, page=(1, slots, 3), pools=int(rng.integers(0, 4)), spread=seed % 5)


@pytest.mark.parametrize("pages", [4095, 4096, 4097, 20000])
def test_fork_over_tiles_of_pages(pages):
    rng = np.random.default_rng(pages)
    table, lengths, refs = sequences(rng, 40, pages, 4, pages // 20, fill=0.9)
    check_fork(table, lengths, refs, rng.integers(-1, 40, 60), rng.integers(0, pages // 20, 60), 4, pools=1, page=(4, 2), width=pages // 20)


def test_fork_many_sequences():
    rng = np.random.default_rng(8)
    table, lengths, refs = sequences(rng, 700, 3000, 2, 6, fill=0.7)
    check_fork(table, lengths, refs, rng.integers(0, 700, 900), rng.integers(0, 3, 900), 2, pools=1, page=(2, 2))


def test_fork_all_from_one_and_none():
    table, lengths, refs = [[4, 2, 0, 1]], [13], [1, 1, 1, 0, 1] + [0] * 30
    check_fork(table, lengths, refs, [0] * 20, [3] * 20, 4, width=5)
    check_fork(table, lengths, refs, [-1] * 3, [0, 9, 0], 4)                # all freed, one starts
    check_fork(table, lengths, refs, [], [], 4)
    check_fork(np.zeros((0, 3)), [], refs, [-1, -1], [5, 0], 4, width=3)
    check_fork(table, lengths, refs, [0, 0], None, 4)
    check_fork([[0, 1]], [8], [1, 1], [0, 0], [0, 0], 4)                    # no part-filled page: nothing to copy


def test_fork_with_too_few_pages():
    table, refs = [[0, 1, -1], [2, 3, -1]], [1, 1, 1, 1, 0, 0]
    r = check_fork(table, [6, 8], refs, [0, 0, 1, 0], [0, 0, 9, 0], 4, width=5)
    assert host(r.status).tolist() == [0, 0, ts.TS_ROW_NO_PAGE, ts.TS_ROW_NO_PAGE] and host(r.lengths).tolist() == [6, 6, 8, 0]
    check_fork(table, [8, 8], refs, [0, 0, 1], [1, 2, 3], 4, width=5)       # the third finds none


def test_fork_bad_rows():
    table = [[0, 1], [9, 2], [3, -1], [4, 5], [1 << 30, 6]]
    check_fork(table, [7, 5, -1, 9, 4], [1, 1, 1, 1, 1, 1, 0, 0], [0, 1, 2, 3, 4, 5, -2], [1] * 7, 4, width=2)
    check_fork([[0, 1, 2]], [12], [1, 1, 1, 0], [0, 0], [0, 0], 4, width=2)  # the new tables are too narrow
    # counts that say less than the tables: pages are free all the same, and nothing breaks
    check_fork([[0, 1], [0, 1]], [8, 8], [1, 1, 0, 0], [0, -1], [1, 5], 4, width=3)


@pytest.mark.parametrize("n,page,dtype,gap", [(70, (5,), "uint8", 0), (65, (2, 16, 8), "bfloat16", 8), (3, (40, 16, 33), "float16", 5),
                                             (2, (200, 128), "float32", 0), (1, (15,), "uint8", 1), (1, (16,), "uint8", 3), (1, (17,), "uint8", 0)])
def test_fork_pools(n, page, dtype, gap):
    rng = np.random.default_rng(n)
    table, lengths, refs = sequences(rng, 6, 40, 4, 8)
    check_fork(table, lengths, refs, rng.integers(0, 6, 12), [1] * 12, 4, pools=n, page=page, dtype=dtype, gap=gap)


# ---------------------------------------------------------------- compact
def check_compact(table, lengths, refs, slots, pools=2, page=(2, 16, 8), dtype="bfloat16", in_place=False, seed=0, gap=0):
    torch = torch_cuda()
    table = np.asarray(table, np.int32)
    banner(f"compact seqs={len(lengths)} pages={len(refs)} slots={slots} width={table.shape[1]} pools={pools}")
    p = [pool_of(len(refs), page, dtype, seed + i, gap) for i in range(pools)]
    before = [raw(x) for x in p]
    t0, r0 = gpu(table), gpu(refs)
    r = ts.ts_pages_compact(t0, gpu(lengths), r0, slots, pools=ts.PagePools(p), in_place=in_place)
    torch.cuda.synchronize()
    o = paged.compact(table.tolist(), list(lengths), refs, slots)
    assert host(r.map).tolist() == o.map
    assert host(r.count).tolist() == [o.count]
    assert host(r.refs).tolist() == o.refs
    assert host(r.table).tolist() == o.table
    assert host(r.status).tolist() == o.status
    if not in_place:
        assert host(r0).tolist() == list(refs) and np.array_equal(host(t0), table)
    for x, b in zip(p, before):
        same(raw(x).ravel(), moved(b, x, o.moves).ravel(), "pool")


@pytest.mark.parametrize("seed", range(16))
def test_compact_random(seed):
    rng = np.random.default_rng(100 + seed)
    pages, slots, seqs = int(rng.integers(1, 400)), int(rng.choice([1, 3, 16])), int(rng.integers(0, 20))
    width = int(rng.integers(1, 40))
    table, lengths, refs = sequences(rng, seqs, pages, slots, width, fill=rng.uniform(0.05, 1.0)) if seqs else ([], [], [0] * pages)
    if seed % 3 == 0:       # pages that no table names are held by something else; others are counted below 0
        for p in rng.integers(0, pages, 5):
            refs[p] += 1
        refs = [-2 if r == 0 and rng.random() < 0.1 else r for r in refs]
    check_compact(np.asarray(table).reshape(seqs, width), lengths, refs, slots, in_place=bool(seed % 2), seed=seed, pools=int(rng.integers(0, 3)),
                  page=(1, slots, 5))


@pytest.mark.parametrize("pages", [4095, 4096, 4097, 8192, 30000])
@pytest.mark.parametrize("fill", [0.1, 0.5, 0.95])
def test_compact_over_tiles_of_pages(pages, fill):
    rng = np.random.default_rng(pages)
    refs = (rng.random(pages) < fill).astype(int).tolist()
    check_compact([[p] for p in np.nonzero(refs)[0][:50]], [1] * 50, refs, 1, pools=1, page=(3, 7), in_place=fill == 0.5)


def test_compact_none_and_all():
    check_compact([[-1]], [0], [0] * 50, 4)
    check_compact([list(range(50))], [200], [1] * 50, 4)
    check_compact([list(range(25, 50))], [100], [0] * 25 + [3] * 25, 4)
    check_compact([[0]], [1], [1], 4)
    check_compact([[0]], [0], [0], 4)


@pytest.mark.parametrize("in_place", [False, True])
def test_compact_bad_rows(in_place):
    check_compact([[5, 1], [9, 3], [-1, 5], [5, 5], [0, 3]], [8, 8, 8, 9, -1], [0, 1, 0, 1, 0, 2, 0, 0], 4, in_place=in_place)


# ---------------------------------------------------------------- copy
def check_copy(source, target, pages, pools=2, page=(2, 16, 8), dtype="bfloat16", seed=0, gap=0):
    torch = torch_cuda()
    banner(f"copy n={len(source)} pages={pages} pools={pools} page={page} {dtype}")
    p = [pool_of(pages, page, dtype, seed + i, gap) for i in range(pools)]
    before = [raw(x) for x in p]
    st = ts.ts_pages_copy(gpu(source), gpu(target), p)
    torch.cuda.synchronize()
    moves, status = paged.copy_pairs(source, target, pages)
    assert host(st).tolist() == status
    for x, b in zip(p, before):
        same(raw(x).ravel(), moved(b, x, moves).ravel(), "pool")


@pytest.mark.parametrize("page,dtype,gap", [((3,), "uint8", 0), ((2, 16, 8), "bfloat16", 4), ((7, 33), "float16", 0), ((64, 16, 128), "float32", 0),
                                            ((16385,), "uint8", 1)])
def test_copy_sizes(page, dtype, gap):
    rng = np.random.default_rng(len(page))
    order = rng.permutation(60)
    check_copy(order[:20].tolist(), order[20:40].tolist(), 60, page=page, dtype=dtype, gap=gap, pools=3)


def test_copy_of_bad_and_repeated_pairs():
    check_copy([0, 1, 2, 3, 4, -1, 9, 8, 1 << 30], [5, 6, 6, 9, 5, 7, 3, 10, 7], 10)
    check_copy([0, 5], [5, 0], 8)                       # a swap is refused
    check_copy([3, 3, 3], [4, 5, 6], 8)                 # one source, several targets
    check_copy([3], [3], 8)
    check_copy([], [], 8)
    rng = np.random.default_rng(0)
    check_copy(rng.integers(0, 40, 1000).tolist(), rng.integers(40, 90, 1000).tolist(), 90, page=(4, 4))


def test_copy_of_more_pools_than_a_launch_takes():
    check_copy([0, 1, 2], [5, 6, 4], 8, pools=130, page=(2, 9))


# ---------------------------------------------------------------- refusals, graphs, streams
def test_refusals_of_the_binding():
    torch = torch_cuda()
    pool = torch.zeros(8, 2, 4, 6, device="cuda")
    i = torch.zeros(2, dtype=torch.int32, device="cuda")
    table, refs = torch.zeros(2, 3, dtype=torch.int32, device="cuda"), torch.zeros(8, dtype=torch.int32, device="cuda")
    for bad in (lambda: ts.PagePools([pool.transpose(1, 2)]), lambda: ts.PagePools([pool, pool[:7]]), lambda: ts.PagePools([pool.cpu()]),
                lambda: ts.PagePools([pool[:, :1].expand(8, 2, 4, 6)]), lambda: ts.ts_pages_fork(table, i, refs[:7], i, 4, pools=[pool]),
                lambda: ts.ts_pages_fork(table.long(), i, refs, i, 4), lambda: ts.ts_pages_fork(table, i, refs.long(), i, 4),
                lambda: ts.ts_pages_fork(table, i[:1], refs, i, 4), lambda: ts.ts_pages_fork(table, i, refs, i, 4, n_new=i[:1]),
                lambda: ts.ts_pages_fork(table, i, refs, i, 0), lambda: ts.ts_pages_fork(table, i, refs, i, 4, width=-1),
                lambda: ts.ts_pages_compact(table, i, refs, 4, pools=[pool[:, 0], pool[:5]]), lambda: ts.ts_pages_compact(table.t(), i, refs, 4),
                lambda: ts.ts_pages_copy(i, i[:1], [pool]), lambda: ts.ts_pages_copy(i, i, []), lambda: ts.ts_pages_copy(i.long(), i, [pool]),
                lambda: ts.ts_cache_append(pool[0], pool[0], i, pool, pool, table, i),
                lambda: ts.ts_cache_append(torch.zeros(1, 2, 6, device="cuda"), torch.zeros(1, 2, 6, device="cuda"), i, pool, pool, table, i),
                lambda: ts.ts_cache_append(torch.zeros(1, 2, 6, device="cuda"), torch.zeros(2, 2, 6, device="cuda"),
                                           torch.zeros(3, dtype=torch.int32, device="cuda"), pool, pool, table, i)):
        with pytest.raises(ts.TopSelectError):
            bad()


def test_captured_step():
    """Grow, append, attend and compact in one graph, replayed on new inputs with eager work between, against eager calls."""
    torch = torch_cuda()
    banner("pages: a captured step")
    rng = np.random.default_rng(5)
    slots, width, pages = 4, 8, 60
    table, lengths, refs = sequences(rng, 6, pages, slots, width, fill=0.5)
    lengths = [min(n, width * slots - 3) for n in lengths]
    refs = [0] * pages
    for row, n in zip(table, lengths):
        for p in row[: -(-n // slots)]:
            refs[p] += 1
    parents = [[0, 0, 1, 2, 5, -1], [5, 4, 3, 2, 1, 0], [1, 1, 1, 1, 1, 1]]
    t, n, r = gpu(table), gpu(lengths), gpu(refs)
    parent, new, offsets = gpu(parents[0]), gpu([2] * 6), gpu(np.arange(7) * 2)
    k, v = (torch.randn(pages, 2, slots, 16, device="cuda") for _ in range(2))
    k0, v0 = k.clone(), v.clone()
    fresh = torch.randn(12, 2, 16, device="cuda")
    q = torch.randn(6, 4, 16, device="cuda")

    def step():
        f = ts.ts_pages_fork(t, n, r, parent, slots, n_new=new, pools=[k, v])
        st = ts.ts_cache_append(fresh, fresh, offsets, k, v, f.table, f.lengths)
        a = ts.ts_cache_attend(q, k, v, f.table, f.lengths)
        c = ts.ts_pages_compact(f.table, f.lengths, f.refs, slots, pools=[k, v])
        b = ts.ts_cache_attend(q, k, v, c.table, f.lengths)
        return [*f, st, a.out, a.lse, a.status, *c, b.out, b.lse, b.status]
    step()
    torch.cuda.synchronize()
    k.copy_(k0), v.copy_(v0)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step()
    for p in parents:
        parent.copy_(gpu(p))
        fresh.mul_(1.5)
        k.copy_(k0), v.copy_(v0)
        want = [x.clone() for x in step()]
        wk, wv = k.clone(), v.clone()
        assert torch.equal(want[5], want[-3])            # attention is the same wherever the pages are
        k.copy_(k0), v.copy_(v0)
        for x in got:
            x.fill_(77)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want)) and torch.equal(k, wk) and torch.equal(v, wv)


def test_decode_with_shared_prompt_and_eviction():
    """A prompt is forked into samples that go on by themselves and end; at each step the attention of every sample is what it
    would be over its own dense cache. Then the weights of a dense cache go to its eviction."""
    torch = torch_cuda()
    banner("pages: decode loop")
    torch.manual_seed(0)
    heads, dim, slots, width, pages, kids = 2, 16, 4, 12, 64, 5
    k, v = (torch.full((pages, heads, slots, dim), float("nan"), device="cuda") for _ in range(2))
    pools = ts.PagePools([k, v])
    table = torch.full((1, width), -1, dtype=torch.int32, device="cuda")
    refs, n = torch.zeros(pages, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    dense = [[torch.empty(0, heads, dim, device="cuda")] * 2]
    parent, grow = [0], 10
    for step in range(16):
        f = ts.ts_pages_fork(table, n, refs, gpu(parent), slots, n_new=gpu([grow] * len(parent)), pools=pools, in_place=True)
        table, n, refs = f.table, f.lengths, f.refs
        fresh = torch.randn(2, len(parent) * grow, heads, dim, device="cuda")
        st = ts.ts_cache_append(fresh[0], fresh[1], gpu(np.arange(len(parent) + 1) * grow), k, v, table, n)
        dense = [[torch.cat([old, fresh[i, c * grow:(c + 1) * grow]]) for i, old in enumerate(dense[p])] for c, p in enumerate(parent)]
        if step % 5 == 4:
            c = ts.ts_pages_compact(table, n, refs, slots, pools=pools, in_place=True)
            assert not host(c.status).any() and int(c.count) == int((refs > 0).sum())
        q = torch.randn(len(parent), 2 * heads, dim, device="cuda")
        a = ts.ts_cache_attend(q, k, v, table, n)
        assert not host(f.status).any() and not host(st).any() and not host(a.status).any()
        for c, (dk, dv) in enumerate(dense):
            s = torch.einsum("hgd,nhd->hgn", q[c].view(heads, 2, dim).double(), dk.double()) / 4
            w = torch.softmax(s, 2)
            want = torch.einsum("hgn,nhd->hgd", w, dv.double()).reshape(2 * heads, dim)
            # 40 positions of 16 dims: (2 * 17 * 14 + 2^3 * 10 + 300) u is less than 1e-4, and |v| < 6
            assert float((a.out[c].double() - want).abs().max()) < 6e-4
        grow = 1
        parent = [0] * kids if step == 0 else list(range(len(parent)))
        if step == 8:
            parent = [2, 0, 0, 4]
    # a dense cache is one page a sequence; its weights decide what stays
    b, budget = 3, 20
    kd, vd = (torch.randn(b, heads, budget + 4, dim, device="cuda") for _ in range(2))
    rows = b * heads
    score, position = torch.zeros(rows, budget + 4, device="cuda"), torch.arange(budget + 4, dtype=torch.int32, device="cuda").repeat(rows, 1)
    ids, full = torch.arange(b, dtype=torch.int32, device="cuda").view(b, 1), torch.full((b,), budget + 4, dtype=torch.int32, device="cuda")
    q = torch.randn(b, 2 * heads, dim, device="cuda")
    a = ts.ts_cache_attend(q, kd, vd, ids, full, weights_slots=budget + 4)
    e = ts.ts_cache_evict(score, position, full.repeat_interleave(heads), torch.full((rows,), budget, dtype=torch.int32, device="cuda"), budget,
                          weights=a.weights.view(rows, 2, budget + 4), k_cache=kd, v_cache=vd, in_place=True)
    assert not host(e.status).any() and not host(a.status).any()
    total = a.weights.view(rows, 2, -1).double().sum(1).float()
    kept = torch.sort(torch.topk(total, budget, dim=1).indices, 1).values
    assert torch.equal(torch.sort(position[:, :budget].long(), 1).values, kept)
    after = ts.ts_cache_attend(q, kd, vd, ids, e.lengths[::heads].contiguous())
    w = a.weights.double().view(rows, 2, -1).gather(2, position[:, :budget].long()[:, None].expand(-1, 2, -1))
    want = (w / w.sum(2, keepdim=True)) @ vd.double().view(rows, -1, dim)[:, :budget]
    assert float((after.out.double().view(rows, 2, dim) - want).abs().max()) < 6e-4


# ---------------------------------------------------------------- caches past one workgroup
@pytest.mark.parametrize("pages,seqs,width,in_place", [(70_000, 40, 30, False), (66_000, 3, 20_000, True), (5000, 1100, 8, False), (9000, 30, 5000, True)])
def test_fork_by_several_launches(pages, seqs, width, in_place):
    rng = np.random.default_rng(pages)
    table, lengths, refs = sequences(rng, seqs, pages, 2, width, fill=0.6)
    n = seqs + 7
    check_fork(table, lengths, refs, rng.integers(-1, seqs, n), rng.integers(0, 5, n), 2, pools=1, page=(4, 2), in_place=in_place)
    parent = np.where(np.arange(n) < seqs, np.arange(n), -1)
    parent[0], parent[1] = -3, seqs
    new = rng.integers(0, max(4, 4 * pages // n), n)                        # more than there are
    new[2] = -1
    check_fork(table, lengths, refs, parent, new, 2, pools=1, page=(4, 2), in_place=in_place)


def test_fork_by_several_launches_with_too_few_pages_for_copies():
    rng = np.random.default_rng(3)
    table, lengths, refs = sequences(rng, 50, 1200, 4, 30, share=0.0, fill=1.0)
    parent = np.sort(rng.integers(0, 50, 1500))
    r = check_fork(table, lengths, refs, parent, np.zeros(1500, int), 4, pools=1, page=(4, 2))
    st = host(r.status)
    assert (st == ts.TS_ROW_NO_PAGE).any() and (st == 0).any()
    table[3][0], table[7][1], lengths[9] = -1, 1 << 30, 1 << 20
    lengths[3], lengths[7] = 8, 8
    check_fork(table, lengths, refs, parent, np.ones(1500, int), 4, pools=1, page=(4, 2))


@pytest.mark.parametrize("pages,seqs,width,in_place", [(20_000, 50, 100, False), (70_000, 20, 300, True), (300, 1100, 20, False), (40_000, 4, 6000, True)])
def test_compact_by_several_launches(pages, seqs, width, in_place):
    rng = np.random.default_rng(pages)
    table, lengths, refs = sequences(rng, seqs, pages, 2, width, fill=0.5)
    table[1][0], lengths[2] = -1, -1
    check_compact(table, lengths, refs, 2, pools=1, page=(3, 7), in_place=in_place)


@pytest.mark.parametrize("pages", [1, 63, 64, 65, 127, 128, 1000, 4096, 16384])
@pytest.mark.parametrize("fill", [0.02, 0.5, 0.97])
def test_compact_at_chunks_of_64_pages(pages, fill):
    rng = np.random.default_rng(pages)
    refs = (rng.random(pages) < fill).astype(int)
    for shift in (0, 64, pages // 2):
        check_compact([[0]], [0], np.roll(refs, shift).tolist(), 1, pools=1, page=(5,), dtype="uint8")
    check_compact([[0]], [0], np.sort(refs).tolist(), 1, pools=1, page=(5,), dtype="uint8")


def test_pools_of_several_page_sizes():
    """Sizes in no order, more of one than a launch takes: every pool is copied once."""
    torch = torch_cuda()
    rng = np.random.default_rng(2)
    sizes = rng.permutation([5] * 70 + [16] * 3 + [300] * 65 + [1, 17, 4096, 40000])
    p = [pool_of(9, (int(n),), "uint8", 50 + i) for i, n in enumerate(sizes)]
    before = [raw(x) for x in p]
    st = ts.ts_pages_copy(gpu([1, 8, 3]), gpu([0, 4, 4]), p)
    torch.cuda.synchronize()
    assert not host(st).any()
    for x, b in zip(p, before):
        same(raw(x).ravel(), moved(b, x, [(1, 0), (3, 4)]).ravel(), "pool")
    before = [raw(x) for x in p]
    refs = [0, 1, 0, 0, 1, 0, 0, 1, 1]
    r = ts.ts_pages_compact(gpu([[1, 4], [7, 8]]), gpu([2, 2]), gpu(refs), 1, pools=p)
    torch.cuda.synchronize()
    assert host(r.table).tolist() == [[1, 0], [2, 3]] and host(r.refs).tolist() == [1, 1, 1, 1, 0, 0, 0, 0, 0]
    for x, b in zip(p, before):
        same(raw(x).ravel(), moved(b, x, [(4, 0), (7, 2), (8, 3)]).ravel(), "pool")


def test_offsets_past_32_bits():
    """Pages of 1 GB, the last of them 5 GB into the pool; slots 5 GB into a cache."""
    torch = torch_cuda()
    banner("pages: 6 GB")
    pool = torch.zeros((6, 1 << 30), dtype=torch.uint8, device="cuda")
    pool[5].view(torch.int32).copy_(torch.arange(1 << 28, dtype=torch.int32, device="cuda"))
    st = ts.ts_pages_copy(gpu([5]), gpu([1]), [pool])
    assert host(st).tolist() == [0] and torch.equal(pool[1], pool[5]) and not bool(pool[0].any()) and not bool(pool[2].any())
    r = ts.ts_pages_compact(gpu([[5, 1]]), gpu([2]), gpu([0, 1, 0, 0, 0, 1]), 1, pools=[pool])
    assert host(r.table).tolist() == [[0, 1]] and torch.equal(pool[0], pool[5])
    pool.zero_()
    k = pool.view(torch.bfloat16).view(6 << 14, 1, 256, 128)                   # pages of 64 KB
    v = torch.zeros_like(k)
    fresh = torch.randn((300, 1, 128), device="cuda").to(torch.bfloat16)
    last = k.shape[0] - 1
    st = ts.ts_cache_append(fresh, fresh, gpu([0, 300]), k, v, gpu([[7, last]]), gpu([400]))
    assert host(st).tolist() == [0]
    for x in (k, v):
        assert torch.equal(torch.cat([x[7, 0, 100:], x[last, 0, :144]]), fresh[:, 0])
        assert not bool(x[last, 0, 144:].any()) and not bool(x[7, 0, :100].any()) and not bool(x[last - 1].any()) and not bool(x[8].any())


# ---------------------------------------------------------------- refused pairs beside sound ones
@pytest.mark.parametrize("pairs", [
    [(1, 6), (-1, 6)], [(1, 6), (1 << 30, 6), (-5, 6)],                  # the later one names no page
    [(1, 5), (5, 5)],                                                    # its source is the first one's target
    [(1, 6), (2, 6), (-1, 6), (3, 6), (-1, 6), (6, 6)],                  # the last sound one of several, not the first
    [(2, 6), (7, 6), (3, 7)],                                            # its source is another target's
    [(-1, 6), (1, 6), (-1, 4), (6, 4), (2, 4)], [(-1, 6), (-1, 6)], [(6, 6), (6, 6), (9, 6)],
    [(1, 1 << 30), (-1, 1 << 30), (2, -1), (3, -1)],
])
def test_copy_of_sound_and_refused_pairs_with_one_target(pairs):
    source, target = zip(*pairs)
    check_copy(list(source), list(target), 9)


@pytest.mark.parametrize("n,pages,bad", [(300, 40, 0.5), (1000, 64, 0.9), (3000, 5000, 0.3), (2000, 9, 0.99)])
def test_copy_of_many_pairs_some_refused(n, pages, bad):
    rng = np.random.default_rng(n)
    half = max(1, pages // 2)
    source, target = rng.integers(0, half, n), rng.integers(half, pages, n)
    wrong = rng.random(n) < bad
    source[wrong] = rng.choice([-1, pages, half, pages - 1], int(wrong.sum()))
    check_copy(source.tolist(), target.tolist(), pages, page=(4, 4), pools=1)


def test_copy_of_a_target_whose_last_sound_pair_comes_early():
    """Behind it stand more refused pairs than a workgroup has threads: out of range, or reading other pairs' targets."""
    for filler in (-1, 7, 6):
        check_copy([1, 2] + [filler] * 700 + [3], [6, 6] + [6] * 700 + [7], 9, page=(4, 4), pools=1)
    check_copy([1] + [7] * 700 + [2] + [8] * 300 + [3, 4], [6] * 1002 + [7, 8], 9, page=(4, 4), pools=1)


# ---------------------------------------------------------------- children that need no page
def test_fork_of_children_without_needs_after_the_pages_ran_out():
    """A token into a part-filled page, nothing new, or no parent at all: no page is needed, so none can be missing."""
    table, refs = [[0, 1, -1], [2, -1, -1], [3, -1, -1]], [1, 1, 1, 1, 0]
    for in_place in (False, True):
        r = check_fork(table, [6, 4, 3], refs, [0, 1, 2, 0, -1, 2, 1], [0, 9, 1, 0, 0, 0, 0], 4, width=5, in_place=in_place)
        assert host(r.status).tolist() == [0, ts.TS_ROW_NO_PAGE, 0, ts.TS_ROW_NO_PAGE, 0, ts.TS_ROW_NO_PAGE, 0]
        assert host(r.lengths).tolist() == [6, 4, 4, 0, 0, 0, 4]
    # no free page at all
    r = check_fork([[0, 1], [2, 3]], [7, 6], [1, 1, 1, 1], [0, 1, -1, -1], [2, 1, 0, 1], 4, width=3)
    assert host(r.status).tolist() == [ts.TS_ROW_NO_PAGE, 0, 0, ts.TS_ROW_NO_PAGE] and host(r.lengths).tolist() == [7, 7, 0, 0]
    # a bad n_new or parent is told as such, also there
    r = check_fork([[0, 1], [2, 3]], [7, 6], [1, 1, 1, 1], [0, 1, 7], [2, -1, 0], 4, width=3)
    assert host(r.status).tolist() == [ts.TS_ROW_NO_PAGE, ts.TS_ROW_BAD_LENGTH, ts.TS_ROW_BAD_PARENT]


def test_fork_of_children_without_needs_by_several_launches():
    """The same for more children than one workgroup takes: a decode step of a pool that is one page short."""
    slots, seqs = 16, 1100
    lengths = np.full(seqs, 20)
    lengths[[3, 500]] = 32                                   # these start a page, the others go on in theirs
    table = np.arange(2 * seqs).reshape(seqs, 2)
    refs = [1] * (2 * seqs) + [0]
    r = check_fork(np.pad(table, ((0, 0), (0, 1)), constant_values=-1), lengths.tolist(), refs, list(range(seqs)) + [-1],
                   [1] * seqs + [0], slots, pools=1, page=(4, 2))
    st = host(r.status)
    assert st[500] == ts.TS_ROW_NO_PAGE and not np.delete(st, 500).any()
    assert (np.delete(host(r.lengths), [3, 500, seqs]) == 21).all()


@pytest.mark.parametrize("seed", range(12))
def test_fork_random_with_few_free_pages(seed):
    """Forks over a pool that is used up, by one workgroup and by several launches."""
    rng = np.random.default_rng(700 + seed)
    seqs = int(rng.integers(2, 30)) if seed % 3 else 1050
    slots, width = int(rng.choice([3, 16])), 6
    table, lengths, refs = sequences(rng, seqs, seqs * 4, slots, width, share=0.2, fill=0.9)
    free = [p for p, r in enumerate(refs) if r == 0]
    for p in free[int(rng.integers(0, 4)):]:
        refs[p] = 1                                          # held by something else
    n = seqs + int(rng.integers(0, 10))
    parent = np.where(rng.random(n) < 0.9, np.arange(n) % seqs, -1)
    check_fork(table, lengths, refs, parent, rng.integers(0, 2, n), slots, width=width + seed % 2, pools=1, page=(4, 2),
               in_place=bool(seed & 1), seed=seed)


# ---------------------------------------------------------------- arguments
@pytest.mark.parametrize("slots", [(1 << 32) + 4, -(1 << 32) + 4, 1 << 31, (1 << 30) + 1, 0, -4])
def test_page_sizes_that_are_none(slots):
    torch = torch_cuda()
    table, refs = gpu([[0, 1], [2, 3]]), gpu([1, 1, 1, 1, 0])
    for call in (lambda: ts.ts_pages_fork(table, gpu([8, 5]), refs, gpu([0, 1]), slots, in_place=True),
                 lambda: ts.ts_pages_compact(table, gpu([8, 5]), refs, slots, in_place=True)):
        with pytest.raises(ts.TopSelectError):
            call()
    torch.cuda.synchronize()
    assert host(refs).tolist() == [1, 1, 1, 1, 0] and host(table).tolist() == [[0, 1], [2, 3]]


def test_append_to_tables_without_columns():
    """Sequences that hold nothing: their tables may have no column, and no new token is the only one that fits."""
    torch = torch_cuda()
    k, v = (torch.zeros(4, 2, 4, 8, device="cuda") for _ in range(2))
    table, fresh = torch.empty((3, 0), dtype=torch.int32, device="cuda"), torch.ones(2, 2, 8, device="cuda")
    assert host(ts.ts_cache_append(fresh[:0], fresh[:0], gpu([0, 0, 0, 0]), k, v, table, gpu([0, 0, 0]))).tolist() == [0, 0, 0]
    st = ts.ts_cache_append(fresh, fresh, gpu([0, 1, 1, 2]), k, v, table, gpu([0, 1, 1]))
    assert host(st).tolist() == [ts.TS_ROW_BAD_LENGTH] * 3 and not bool(k.any()) and not bool(v.any())
