"""GPU tests of ts_token_logp against the binary64 oracle.

Tolerance, from the arithmetic (u = 2^-24, L = ln V): the base-2 exponent (x - m) * c carries three roundings (the
difference, c, the product), so a term exp(d) is off by at most (3 |d| + 2) u relative (the hardware exponential within
one ulp, 2 u), and nine additions of a thread's 32 terms in four chains add 9 u. The p-weighted mean of |d| is at most
the entropy, so at most L, and of d^2 at most L^2 + 1 (the second moment of -ln p of any V outcomes). Hence log S is
off by at most (3 L + 11) u, and sum exp(d) d / S by (3 (L^2 + 1) + 13 L) u plus L times the error of S. What is left
is binary64; each output is rounded once (u relative).
"""
import math

import numpy as np
import pytest

import oracle
import top_select_gumbel_amd as ts
from gpu_helpers import banner, host, torch_cuda

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
TYPES = ["float32", "bfloat16", "float16"]


def tol_log_s(v):
    return (3 * math.log(max(v, 2)) + 11) * U


def tol_entropy(v):
    big = math.log(max(v, 2))
    return tol_log_s(v) * (1 + big) + (3 * (big * big + 1) + 13 * big) * U


def make(rows, v, dtype, seed, scale=3.0, pad=0, shift=0):
    """Logits of `dtype`, rows `v + pad` apart, starting `shift` elements into their buffer."""
    torch = torch_cuda()
    rng = np.random.default_rng(seed)
    flat = torch.from_numpy((rng.standard_normal(shift + rows * (v + pad)) * scale).astype(np.float32)).to(getattr(torch, dtype))
    return flat.cuda()[shift:].view(rows, v + pad)[:, :v]


def i32(a):
    return torch_cuda().tensor(np.asarray(a, np.int32)).cuda()


def f32(a):
    return None if a is None else torch_cuda().tensor(np.asarray(a, np.float32)).cuda()


def check(x, tokens, t, n_top, label="", rows=None, res=None):
    torch = torch_cuda()
    banner(f"token_logp {label} {tuple(x.shape)} {x.dtype} n_top={n_top}")
    if res is None:
        res = ts.ts_token_logp(x, None if tokens is None else i32(tokens), f32(t), n_top=n_top)
    torch.cuda.synchronize()
    xs = x.double().cpu().numpy()
    got = {k: None if v is None else host(v) for k, v in res._asdict().items()}
    v = x.shape[1]
    for r in range(x.shape[0]) if rows is None else rows:
        token = -1 if tokens is None else int(tokens[r])
        tv = 1.0 if t is None else oracle.to_f32(t[r])
        o = oracle.token_logp_row(xs[r], tv, token, n_top)
        where = f"{label} row {r}"
        assert got["status"][r] == o.status, where

        def near(a, b, tol):
            a = float(a)
            if abs(b) >= 2.0 ** 128 * (1 - 2.0 ** -25):   # past half a step above the largest fp32: rounds to infinity
                b = math.copysign(math.inf, b)
            if not math.isfinite(b):
                assert a == b or (math.isnan(a) and math.isnan(b)), (where, a, b)
            else:
                assert abs(a - b) <= tol + U * abs(b), (where, a, b, abs(a - b), tol)
        near(got["lse"][r], o.lse, tol_log_s(v))
        near(got["entropy"][r], o.entropy, tol_entropy(v))
        if tokens is not None:
            near(got["logp"][r], o.logp, tol_log_s(v))
            assert got["rank"][r] == o.rank, (where, got["rank"][r], o.rank)
        if n_top:
            assert got["top_idx"][r].tolist() == o.top_idx, where
            for a, b in zip(got["top_logp"][r], o.top_logp):
                near(a, b, tol_log_s(v))
    return got


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("v", [1, 2, 3, 7, 8, 9, 31, 255, 1000, 8191, 8192, 8193, 8200, 16385, 50001])
def test_sizes(v, dtype):
    rng = np.random.default_rng(v)
    rows = 5 if v < 10000 else 3
    x = make(rows, v, dtype, v, pad=v % 3, shift=v % 5)
    tokens = rng.integers(0, v, rows)
    tokens[0] = int(x[0].float().argmax())
    tokens[-1] = -1
    for n_top, t in [(0, None), (1, None), (5, rng.uniform(0.5, 1.5, rows)), (64, None)]:
        check(x, tokens, t, n_top, "sizes")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("v", [40, 8192, 20011])
def test_ties(v, dtype):
    rng = np.random.default_rng(v + 1)
    torch = torch_cuda()
    x = torch.from_numpy(rng.integers(-2, 3, (6, v)).astype(np.float32))
    x[1] = 0.25                                    # all equal: the lowest ids, found exactly
    x[2] = torch.where(x[2] == 0, torch.tensor(-0.0), x[2])
    x[2, ::3] = 0.0                                # -0 and +0 are one value
    x[3, v // 2:] = 2.0
    x[4] = torch.finfo(getattr(torch, dtype)).min   # the type's lowest value is a logit like others
    x[5, : v - 5] = torch.finfo(getattr(torch, dtype)).min
    x = x.to(getattr(torch, dtype)).cuda()
    for n in (1, 20, 64):
        check(x, rng.integers(0, v, 6), None, n, "ties")
    check(x, np.full(6, v - 1), None, 3, "ties, last token")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("v", [70, 100, 200, 700, 8192, 8300, 20011])
def test_alternatives_among_neighbours(v, dtype):
    """Short rows, and masks that leave a run of neighbours: the candidates sit in few threads, several in each."""
    rng = np.random.default_rng(v + 7)
    live = [65, 100, 130, 300, 600, 1500]
    x = make(len(live) + 2, v, dtype, v + 8)
    for r, m in enumerate(live):
        at = int(rng.integers(0, max(v - m, 1)))
        x[r, :at] = -math.inf
        x[r, at + m:] = -math.inf
    x[len(live)] = x[len(live)].sort().values          # the large ones in the last threads
    for n in (1, 5, 20, 64):
        check(x, rng.integers(0, v, x.shape[0]), None, n, "neighbours")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("v", [33, 9000])
def test_masked_and_rejected_rows(v, dtype):
    rng = np.random.default_rng(v + 2)
    x = make(14, v, dtype, v)
    x[0, :] = -math.inf                            # nothing left
    x[1, 1:] = -math.inf                           # one token left
    x[2, : v - 1] = -math.inf
    x[3, rng.random(v) < 0.9] = -math.inf
    x[4, 5] = math.nan
    x[5, :] = math.nan
    x[6, v - 1] = math.inf
    x[7, 3], x[7, 4] = math.nan, -math.inf
    x[8, :] = -math.inf
    x[8, 2] = math.inf
    x[9, : v // 2] = -math.inf
    x[9, 7] = math.nan                              # among masked places
    tokens = rng.integers(0, v, 14)
    tokens[1], tokens[2], tokens[3] = 0, 0, int(np.nonzero(np.isneginf(x[3].float().cpu().numpy()))[0][0])
    tokens[10], tokens[11], tokens[12], tokens[13] = -1, v, -2, 2 ** 31 - 1
    for n in (0, 4, 64):
        got = check(x, tokens, None, n, "masked")
    assert got["status"].tolist() == [1, 0, 0, 0, 1, 1, 1, 1, 1, 1, 0, 6, 6, 0 if v > 2 ** 31 - 1 else 6]


def test_negative_nan_is_seen():
    torch = torch_cuda()
    x = torch.zeros(4, 100, dtype=torch.float32)
    x.view(torch.int32)[:2, 17] = -1               # a NaN with its sign bit set
    xb = x.bfloat16()
    xb.view(torch.int16)[:2, 17] = -1
    for y in (x.cuda(), xb.cuda()):
        assert host(ts.ts_token_logp(y, i32([0] * 4)).status).tolist() == [1, 1, 0, 0]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("v", [50, 8500])
def test_temperatures(v, dtype):
    t = [1e-3, 100.0, 0.0, 0.0, 3e38, 1e-38, 1e-45, 2.0 ** -100, math.nan, -1.0, math.inf, -0.0]
    x = make(len(t), v, dtype, v + 3)
    tokens = x.float().argmax(1).cpu().numpy()
    tokens[3] = (tokens[3] + 1) % v
    tokens[0] = 1
    rng = np.random.default_rng(v)
    # at the smallest temperatures lse = m / T overflows fp32, as its definition does
    rows = [0, 1, 2, 3, 4, 8, 9, 10, 11]
    got = check(x, tokens, t, 6, "temperatures", rows=rows)
    for r in (5, 6, 7):                             # as good as greedy
        assert got["status"][r] == 0 and got["logp"][r] == 0.0 and got["rank"][r] == 1 and got["entropy"][r] == 0.0
    bad = make(3, v, dtype, v)
    bad[0, 0] = math.nan                            # status precedence: logits, temperature, token
    assert host(ts.ts_token_logp(bad, i32([v, v, v]), f32([-1.0, -1.0, 1.0])).status).tolist() == [1, 4, 6]


def test_wide_range_of_magnitudes():
    # maxima and distances that overflow a product with 1/T, and distances beyond fp32
    x = np.full((4, 9000), -3e38, np.float32)
    x[0, 100], x[0, 200] = 3e38, 2.9e38
    x[1, 100], x[1, 200] = 1e30, 1e30
    x[2, :] = np.linspace(-1e4, 1e4, 9000)
    x[3, :] = np.linspace(-1e-30, 1e-30, 9000)
    torch = torch_cuda()
    check(torch.from_numpy(x).cuda(), [100, 200, 8999, 0], [1.0, 1e-6, 50.0, 1e-30], 3, "magnitudes")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("v", [6, 8192, 20011, 60000])
def test_confident_rows_keep_their_small_log_probabilities(v, dtype):
    # one token far above equal others: logp = -log1p((v - 1) exp(-d)), whose terms carry (3 d + 2) u and whose fp32 sums 9 u
    # more; with the output's rounding the relative error is at most (3 d + 12) u. S itself is a binary64 number from 1 to 2,
    # rounded in the tile, in its join with the others (a product and a sum each) and in the logarithm: at most 5 times
    # 2^-53, absolutely, which only logp below 1e-9 feels
    torch = torch_cuda()
    gaps, t = [4.0, 9.0, 12.0, 16.0, 20.0, 24.0], 0.75
    x = torch.full((len(gaps), v), 1.25)
    where = [0, v - 1, v // 2, min(8191, v - 1), min(8192, v - 1), 1]
    for r, (g, at) in enumerate(zip(gaps, where)):
        x[r, at] = 1.25 + g
    x = x.to(getattr(torch, dtype)).cuda()
    for tv in (1.0, t):
        r = ts.ts_token_logp(x, i32(where), f32([tv] * len(gaps)), n_top=1)
        for i, g in enumerate(gaps):
            d = float(x[i, where[i]].double() - 1.25) / oracle.to_f32(tv)
            want = -math.log1p((v - 1) * math.exp(-d))
            for got in (float(r.logp[i]), float(r.top_logp[i, 0])):
                assert abs(got - want) <= (3 * d + 12) * U * abs(want) + 5 * 2.0 ** -53, (i, got, want)


@pytest.mark.parametrize("v,dtype", [(151936, "float32"), (128256, "bfloat16"), (300007, "float16")])
def test_long_rows(v, dtype):
    rng = np.random.default_rng(9)
    x = make(4, v, dtype, 9)
    x[1] = x[1].sort(descending=True).values        # the best all in one tile
    x[2] = x[2].sort().values
    x[3] = 1.0                                      # every tile finds its lowest ids exactly
    check(x, rng.integers(0, v, 4), rng.uniform(0.5, 1.5, 4), 64, "long")
    check(x, rng.integers(0, v, 4), None, 20, "long")


@pytest.mark.parametrize("v,dtype", [(262144, "float32"), (1200007, "bfloat16"), (2500001, "float16")])
def test_alternatives_of_the_longest_rows(v, dtype):
    """More candidates than one wave takes at a time, in several shares; ties in all of them."""
    torch = torch_cuda()
    x = make(3, v, dtype, v + 3)
    x[1] = torch.from_numpy(np.random.default_rng(v).integers(0, 3, v).astype(np.float32)).to(x.dtype).cuda()
    x[2, 20000:] = torch.sort(x[2, 20000:]).values      # the large ones in the last tiles
    for n in (5, 20, 64):
        check(x, [7, v - 1, -1], None, n, "longest rows")


def test_outputs_are_optional_and_nothing_else_is_written():
    torch = torch_cuda()
    x = make(3, 9001, "float32", 4)
    full = ts.ts_token_logp(x, i32([1, 2, 3]), None, n_top=3, want_stats=True)
    none = ts.ts_token_logp(x)
    assert none.logp is None and none.rank is None and none.top_idx is None and none.stats is None
    assert torch.equal(none.lse, full.lse) and torch.equal(none.entropy, full.entropy)
    less = ts.ts_token_logp(x, i32([1, 2, 3]), want_rank=False, want_entropy=False, want_lse=False)
    assert less.rank is None and less.entropy is None and less.lse is None and torch.equal(less.logp, full.logp)
    m, s = host(x.max(1).values), host(full.stats)
    assert np.array_equal(s[:, 0], m) and (s[:, 1] >= 1).all()
    empty = ts.ts_token_logp(x[:0], i32([]), n_top=2)
    assert empty.logp.shape == (0,) and empty.top_idx.shape == (0, 2)


@pytest.mark.parametrize("dtype", TYPES)
def test_same_bits_whatever_the_batch(dtype):
    torch = torch_cuda()
    v = 20011
    x = make(7, v, dtype, 21)
    tokens, t = i32([3, 4, 5, 6, 7, 8, 9]), f32([1, 0.7, 1.3, 1, 0.9, 2, 1])
    whole = ts.ts_token_logp(x, tokens, t, n_top=9, want_stats=True)
    for r in range(7):
        for shift in (0, 1, 3):                     # another address, another batch
            buf = torch.zeros(2 * v + 64, dtype=x.dtype, device="cuda")
            y = buf[shift:shift + 2 * (v + 5)].view(2, v + 5)[:, :v]
            y[1] = x[r]
            one = ts.ts_token_logp(y, i32([0, int(tokens[r])]), f32([1.0, float(t[r])]), n_top=9, want_stats=True)
            for a, b in zip(one, whole):
                assert torch.equal(a[1], b[r]), (r, shift)


def test_streams_and_graphs():
    torch = torch_cuda()
    x = make(40, 60000, "bfloat16", 30)
    y = make(40, 60000, "bfloat16", 31)
    tokens = i32(np.arange(40))
    want = [ts.ts_token_logp(z, tokens, n_top=8) for z in (x, y)]
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for z, s in ((x, s1), (y, s2)) * 3:              # calls at once on two streams
        with torch.cuda.stream(s):
            got.append(ts.ts_token_logp(z, tokens, n_top=8))
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(g[:6], want[i % 2][:6]))
    graphs = []
    src = [x.clone(), y.clone()]
    for z in src:                                    # two graphs, replayed at once
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = ts.ts_token_logp(z, tokens, n_top=8)
        graphs.append((g, out))
    for k in range(4):
        for z, w in zip(src, (x, y) if k % 2 == 0 else (y, x)):
            z.copy_(w)
        torch.cuda.synchronize()
        for (g, _), s in zip(graphs, (s1, s2)):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        torch.zeros(1000, device="cuda").add_(1).sum().item()
        for (_, out), w in zip(graphs, want if k % 2 == 0 else want[::-1]):
            assert all(torch.equal(a, b) for a, b in zip(out[:6], w[:6])), k


def test_binding_refusals():
    torch = torch_cuda()
    x = make(2, 64, "float32", 1)
    for bad in (lambda: ts.ts_token_logp(x.double(), i32([0, 0])), lambda: ts.ts_token_logp(x.t(), i32([0] * 64)),
                lambda: ts.ts_token_logp(x[0], i32([0])), lambda: ts.ts_token_logp(x, i32([0])),
                lambda: ts.ts_token_logp(x, torch.zeros(2, dtype=torch.int64, device="cuda")),
                lambda: ts.ts_token_logp(x, torch.zeros(2, dtype=torch.int32)),
                lambda: ts.ts_token_logp(x, i32([0, 0]), torch.ones(2, dtype=torch.float64, device="cuda")),
                lambda: ts.ts_token_logp(x, i32([0, 0]), n_top=65), lambda: ts.ts_token_logp(x.expand(2, 64)[:, ::2], i32([0, 0])),
                lambda: ts.ts_token_logp(x[:1].expand(3, 64), i32([0] * 3))):
        with pytest.raises(ts.TopSelectError):
            bad()


@pytest.mark.parametrize("v", [100, 20000])
def test_empty_batch(v):
    torch = torch_cuda()
    x, tokens = torch.empty((0, v), device="cuda"), torch.empty(0, dtype=torch.int32, device="cuda")
    r = ts.ts_token_logp(x, tokens, n_top=5, want_stats=True)
    assert [tuple(t.shape) for t in r] == [(0,), (0,), (0,), (0,), (0, 5), (0, 5), (0, 4), (0,)]
    assert ts.ts_token_logp_backward(x, tokens, None, r.stats).shape == (0, v)
    r = ts.ts_token_logp(x, want_entropy=False, want_lse=False)
    assert all(t is None for t in r[:-1]) and r.status.shape == (0,)
