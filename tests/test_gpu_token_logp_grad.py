"""GPU tests of ts_token_logp_backward against the binary64 oracle's formula and against differences.

Tolerance, from the arithmetic (u = 2^-24, L = ln V): exp(d) is off by at most (3 |d| + 2) u relative, S and its fp32
copy by (3 L + 12) u, D by the entropy's tolerance, and forming q, k0, k1 and the product takes at most sixteen more
roundings of u. So element i is off by at most
  (p_i / T) ((|l - a| + |h| (|d_i| + |D|)) (3 |d_i| + 3 L + 30) u + |h| tol_D) + 3 u |a| / T at the token,
plus half a step of the logits' type (eps / 2 relative; 2^-25 in fp16's subnormal range).
"""
import math

import numpy as np
import pytest

import oracle
import top_select_gumbel_amd as ts
from gpu_helpers import banner, host, torch_cuda
from test_gpu_token_logp import TYPES, U, f32, i32, make, tol_entropy

pytestmark = pytest.mark.gpu


def run(x, tokens, t, a, h, l, out=None):
    ti, tf = None if tokens is None else i32(tokens), f32(t)
    fwd = ts.ts_token_logp(x, ti, tf, want_rank=False, want_stats=True)
    g = ts.ts_token_logp_backward(x, ti, tf, fwd.stats, f32(a), f32(h), f32(l), out=out)
    torch_cuda().cuda.synchronize()
    return fwd, g


def check(x, tokens, t, a, h, l, label="", g=None):
    torch = torch_cuda()
    banner(f"token_logp_backward {label} {tuple(x.shape)} {x.dtype}")
    if g is None:
        _, g = run(x, tokens, t, a, h, l)
    assert g.dtype == x.dtype and g.shape == x.shape
    half = torch.finfo(x.dtype).eps / 2
    floor = 2.0 ** -25 if x.dtype == torch.float16 else 2.0 ** -126
    xs, gs = x.double().cpu().numpy(), g.double().cpu().numpy()
    v = x.shape[1]
    for r in range(x.shape[0]):
        token = -1 if tokens is None else int(tokens[r])
        tv = 1.0 if t is None else oracle.to_f32(t[r])
        av, hv, lv = (0.0 if q is None else oracle.to_f32(q[r]) for q in (a, h, l))
        want = oracle.token_logp_grad_row(xs[r], tv, token, av, hv, lv)
        av = av if token >= 0 else 0.0
        d = np.maximum((xs[r] - xs[r].max()) / tv, -2000.0)
        p = np.exp(d)
        p /= p.sum()
        mean = abs((p * d).sum())
        tol = p / tv * ((abs(lv - av) + abs(hv) * (abs(d) + mean)) * (3 * abs(d) + 3 * math.log(max(v, 2)) + 30) * U
                        + abs(hv) * tol_entropy(v))
        if token >= 0:
            tol[token] += 3 * U * abs(av) / tv
        tol = tol * (1 + half) + half * abs(want) + floor
        bad = np.nonzero(~(abs(gs[r] - want) <= tol))[0]
        assert not len(bad), (label, r, bad[:5], gs[r][bad[:5]], want[bad[:5]], tol[bad[:5]])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("v", [1, 2, 7, 8, 9, 100, 8191, 8192, 8193, 20011])
def test_sizes(v, dtype):
    rng = np.random.default_rng(v)
    rows = 4
    x = make(rows, v, dtype, v, pad=v % 4, shift=v % 3)
    tokens = rng.integers(0, v, rows)
    tokens[1] = -1
    a, h, l = rng.standard_normal((3, rows))
    check(x, tokens, None, a, None, None, "logp")
    check(x, tokens, rng.uniform(0.5, 1.5, rows), a, h, l, "all")
    check(x, None, None, None, h, None, "entropy")
    check(x, None, None, None, None, l, "lse")
    check(x, tokens, None, None, None, None, "nothing")
    # a batch whose tokens are the same index, first and last
    check(x, np.full(rows, v - 1), None, a, h, None, "last token")
    check(x, np.zeros(rows, int), None, a, h, None, "first token")


@pytest.mark.parametrize("dtype", TYPES)
def test_masks_and_peaks(dtype):
    torch = torch_cuda()
    v = 8300
    rng = np.random.default_rng(5)
    x = make(7, v, dtype, 6)
    x[0, rng.random(v) < 0.99] = -math.inf
    x[1, 1:] = -math.inf
    x[2, 4000] = 60.0                              # nearly all weight on one token
    x[3, :] = torch.finfo(x.dtype).min
    x[3, 10:12] = 1.0
    x[4, : v // 2] = torch.finfo(x.dtype).min
    x[5, :] = 0.5
    a, h, l = rng.standard_normal((3, 7))
    tokens = [int(x[0].float().argmax()), 0, 4000, 11, 5, 8299, -1]
    check(x, tokens, [1.0, 0.5, 1.0, 2.0, 1.0, 1.0, 0.7], a, h, l, "masks")
    g = host(run(x, tokens, None, a, h, l)[1].float())
    assert not g[0][np.isneginf(host(x[0].float()))].any() and not g[1][1:].any()   # row 1's one live token: a + (l - a)
    # the gradient of a masked given token: the formula's
    masked = int(np.nonzero(np.isneginf(host(x[0].float())))[0][0])
    check(x[:1], [masked], None, [1.5], None, None, "masked token")


def test_rejected_and_greedy_rows():
    x = make(8, 9000, "float32", 8)
    x[0, 3] = math.nan
    x[1, :] = -math.inf
    tokens, t = [1, 1, 9000, -5, 1, 2, 3, -1], [1, 1, 1, 1, -1.0, 0.0, 1, 0.0]
    _, g = run(x, tokens, t, np.ones(8), np.ones(8), np.ones(8))
    g = host(g)
    assert np.isnan(g[:5]).all() and not g[5].any() and np.isfinite(g[6]).all() and not g[7].any()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("v", [5, 9001])
def test_in_place_and_strided_output(v, dtype):
    torch = torch_cuda()
    rng = np.random.default_rng(3)
    x = make(5, v, dtype, 12, pad=3, shift=1)
    a, h, l = rng.standard_normal((3, 5))
    tokens = rng.integers(0, v, 5)
    _, want = run(x, tokens, None, a, h, l)
    big = torch.full((5, v + 9), 7.0, dtype=x.dtype, device="cuda")
    _, got = run(x, tokens, None, a, h, l, out=big[:, 3:3 + v])
    assert torch.equal(got, want)
    assert (big[:, :3] == 7).all() and (big[:, 3 + v:] == 7).all()        # nothing beside the rows is written
    y = x._base[1:].view(5, v + 3) if x._base is not None else x
    pad_before = y[:, v:].clone()
    _, same = run(x, tokens, None, a, h, l, out=x)
    assert same.data_ptr() == x.data_ptr() and torch.equal(x, want) and torch.equal(y[:, v:], pad_before)
    with pytest.raises(ts.TopSelectError):
        run(x[1:], tokens[1:], None, a[1:], h[1:], l[1:], out=x[:-1])


def test_against_differences_of_the_forward_call():
    # fp32 logits near 1: a central difference with step 2^-6 in fp32 outputs (steps are exact); its own error is the
    # truncation step^2 / 6 times a third derivative below 1, 4.1e-5 times |gradients| (sum below 3), and the two forward
    # values' tolerance (below 5e-6 at this size, |value| below 8) over 2 step, 1.6e-4 each way
    torch = torch_cuda()
    v, step = 12, 2.0 ** -6
    rng = np.random.default_rng(1)
    base = rng.integers(-64, 65, v).astype(np.float32) / 32
    a, h, l = np.float32(1.0), np.float32(0.5), np.float32(-0.25)
    x = np.stack([base] + [base + s * step * (np.arange(v) == i) for i in range(v) for s in (1, -1)]).astype(np.float32)
    n = len(x)
    fwd, g = run(torch.from_numpy(x).cuda(), [4] * n, [1.5] * n, [a] * n, [h] * n, [l] * n)
    loss = a * host(fwd.logp).astype(np.float64) + h * host(fwd.entropy) + l * host(fwd.lse)
    diff = (loss[1::2] - loss[2::2]) / (2 * step)
    assert np.abs(diff - host(g)[0]).max() <= 3 * step * step / 6 + 2 * 5e-6 / (2 * step) * 1.75


def test_graph_and_streams():
    torch = torch_cuda()
    x = make(64, 33000, "bfloat16", 40)
    tokens, a = i32(np.arange(64)), f32(np.ones(64))
    def step(z):
        f = ts.ts_token_logp(z, tokens, want_rank=False, want_stats=True)
        return f.logp, ts.ts_token_logp_backward(z, tokens, None, f.stats, a, a)
    want = step(x)
    torch.cuda.synchronize()
    src = torch.zeros_like(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(src)
    for k in range(3):
        src.copy_(x if k != 1 else x.flip(0))
        graph.replay()
        torch.cuda.synchronize()
        torch.ones(1000, device="cuda").cumsum(0).sum().item()
        if k != 1:
            assert all(torch.equal(p, q) for p, q in zip(out, want)), k
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = step(x)
    s.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got, want))


def test_refusals():
    torch = torch_cuda()
    x = make(2, 64, "float32", 1)
    st = ts.ts_token_logp(x, i32([0, 1]), want_stats=True).stats
    for bad in (lambda: ts.ts_token_logp_backward(x, i32([0, 1]), None, st[:1], f32([1, 1])),
                lambda: ts.ts_token_logp_backward(x, i32([0, 1]), None, None, f32([1, 1])),
                lambda: ts.ts_token_logp_backward(x, None, None, st, f32([1, 1])),
                lambda: ts.ts_token_logp_backward(x, i32([0, 1]), None, st, f32([1])),
                lambda: ts.ts_token_logp_backward(x, i32([0, 1]), None, st, torch.ones(2, device="cuda").half()),
                lambda: ts.ts_token_logp_backward(x, i32([0, 1]), None, st, f32([1, 1]), out=torch.empty(2, 64, device="cuda").half()),
                lambda: ts.ts_token_logp_backward(x, i32([0, 1]), None, st, f32([1, 1]), out=torch.empty(2, 63, device="cuda")),
                lambda: ts.ts_token_logp_backward(x, i32([0, 1]), None, st, f32([1, 1]), out=torch.empty(2, 64))):
        with pytest.raises(ts.TopSelectError):
            bad()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("v,gap", [(5, 0), (100, 0), (9001, 3)])
def test_gradient_rows_between_the_logits_rows(v, gap, dtype):
    """Logits and gradient in one buffer, row by row: their address spans intersect, their rows do not."""
    torch = torch_cuda()
    rng = np.random.default_rng(v)
    rows, width = 6, 2 * (v + gap)
    x = make(rows, v, dtype, v + 17)
    a, h, l = rng.standard_normal((3, rows))
    tokens = rng.integers(0, v, rows)
    _, want = run(x, tokens, None, a, h, l)
    for first in (True, False):                     # the gradient behind and before each row's logits
        buf = torch.full((rows, width), 7.0, dtype=x.dtype, device="cuda")
        xs, gs = (buf[:, :v], buf[:, v + gap:2 * v + gap]) if first else (buf[:, v + gap:2 * v + gap], buf[:, :v])
        xs.copy_(x)
        _, got = run(xs, tokens, None, a, h, l, out=gs)
        assert torch.equal(got, want) and torch.equal(xs, x)
        assert (buf[:, v:v + gap] == 7).all() and (buf[:, 2 * v + gap:] == 7).all()
    lower = torch.zeros(2 * rows, v, dtype=x.dtype, device="cuda")      # one row down, every second row
    lower[::2].copy_(x)
    _, got = run(lower[::2], tokens, None, a, h, l, out=lower[1::2])
    assert torch.equal(got, want) and torch.equal(lower[::2], x)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("v", [100, 9001, 60000])
def test_gradients_at_large_temperatures(v, dtype):
    # 1 / (T S) is below the smallest normal number, the gradient, of incoming ones about as large as T, is not
    torch = torch_cuda()
    rng = np.random.default_rng(v)
    t = [2.0 ** 64, 2.0 ** 65, 1e30, 1e36, 1e38, 3e38]
    x = torch.from_numpy((rng.standard_normal((len(t), v)) * np.array(t)[:, None] * 0.1).astype(np.float32)).to(getattr(torch, dtype)).cuda()
    a, h, l = rng.standard_normal((3, len(t))) * np.array(t) * [[0.3], [0.01], [0.1]]
    check(x, rng.integers(0, v, len(t)), t, a, None, l, "large T")
    check(x, rng.integers(0, v, len(t)), t, a, h, l, "large T, entropy")


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("v", [6, 9001])
def test_distances_beyond_the_largest_number(v, dtype):
    # x - m is below the lowest fp32, (x - m) / T a few units: such logits have weight
    torch = torch_cuda()
    rng = np.random.default_rng(v)
    x = torch.from_numpy((rng.uniform(-3e38, 3e38, (3, v))).astype(np.float32))
    x[:, 1], x[:, 3] = 3.2e38, -3.2e38
    x[2] = -3.2e38
    x[2, 1] = 3.2e38
    x = x.to(getattr(torch, dtype)).cuda()
    t = [1e38, 6e37, 1.5e38]
    # gradients of about 1e38, so that p g / T is a few hundredths
    check(x, [3, 1, 2], t, [1e38, -2e37, 3e37], None, [1e37, 0.0, 2e37], "far apart")
    check(x, [3, 1, 2], t, [1e38, 1e37, 1e37], [1e36, -2e36, 1e36], None, "far apart, entropy")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("v", [6, 8192, 20011, 60000])
def test_confident_rows_keep_the_given_tokens_gradient(v, dtype):
    # one token far above equal others, and given: its gradient is a (1 - p) / T = a (S - 1) / (S T). S - 1 has terms off by
    # (3 d + 2) u and fp32 sums that add 9 u, as the forward call's test says. (S - 1) / S is formed in binary64, where S is off by
    # at most 4 times 2^-53, and rounded to fp32 (u); 1 / T and two products add 3 u: (3 d + 15) u. That holds where S < 4/3;
    # above, nothing much cancels and the general tolerance is the bound
    torch = torch_cuda()
    gaps = [4.0, 9.0, 12.0, 16.0, 20.0, 24.0]
    x = torch.full((len(gaps), v), 1.25)
    where = [0, v - 1, v // 2, min(8191, v - 1), min(8192, v - 1), 1]
    for r, (g, at) in enumerate(zip(gaps, where)):
        x[r, at] = 1.25 + g
    x = x.to(getattr(torch, dtype)).cuda()
    a = [1.0, -0.7, 1.3, -1.0, 0.9, 2.5]
    half = torch.finfo(x.dtype).eps / 2
    floor = 2.0 ** -25 if dtype == "float16" else 0.0
    for tv in (1.0, 0.75):
        t = None if tv == 1.0 else [tv] * len(gaps)
        check(x, where, t, a, None, None, "confident")
        check(x, where, t, a, [0.3, -0.2, 1.0, 0.1, -1.0, 0.5], [1.0, 0.1, 1.3, 0.0, -0.9, 0.2], "confident, all")
        g = run(x, where, t, a, None, None)[1].double().cpu().numpy()
        sharp = 0
        for i in range(len(gaps)):
            d, av = float(x[i, where[i]].double() - 1.25) / tv, oracle.to_f32(a[i])
            rest = (v - 1) * math.exp(-d)
            if rest >= 0.333:
                continue
            sharp += 1
            want = av * rest / (1 + rest) / tv
            tol = (3 * d + 15) * U * abs(want) + 4 * 2.0 ** -53 * abs(av) / tv
            assert abs(g[i, where[i]] - want) <= tol * (1 + half) + half * abs(want) + floor, (tv, i, g[i, where[i]], want)
        assert sharp >= 3


def test_confident_rows_at_the_largest_and_smallest_temperatures():
    # the same at a temperature that is scaled and one that acts as 2^-100, for greedy and for rejected rows
    x = np.full((5, 50), -3e38, np.float32)
    x[:, 7] = 3e38
    x[1] = -1e-30
    x[1, 7] = 1e-30
    t = [2e37, 1e-35, 2e37, np.nan, 0.0]
    a = [1e37, 1.0, 1e37, 1.0, 1.0]
    xt = torch_cuda().from_numpy(x).cuda()
    tokens = [7, 7, 50, 7, 7]
    g = host(run(xt, tokens, t, a, None, None)[1])
    assert np.isnan(g[2]).all() and np.isnan(g[3]).all() and not g[4].any()
    d = 2 * oracle.to_f32(3e38) / oracle.to_f32(2e37)
    rest = 49 * math.exp(-d)
    want = oracle.to_f32(1e37) / oracle.to_f32(2e37) * rest / (1 + rest)
    assert rest < 1e-11 and abs(g[0, 7] - want) <= (3 * d + 15) * U * want + 4 * 2.0 ** -53
    p = 1 / (1 + 49 * math.exp(-2 * oracle.to_f32(1e-30) * 2.0 ** 100))     # 2.5 away
    want = (1 - p) * 2.0 ** 100
    assert 0.15 < p < 0.3 and abs(g[1, 7] - want) <= want * 90 * U
    g = host(run(xt, tokens, t, a, None, a)[1])       # l = a: what is left is a / T
    assert abs(g[0, 7] - oracle.to_f32(1e37) / oracle.to_f32(2e37)) <= 3 * U
    assert abs(g[1, 7] - 2.0 ** 100) <= 2.0 ** 100 * 90 * U


def test_confident_row_whose_backward_call_is_invalid():
    # the forward call's statistics are in order, the backward call's token or temperature is not
    x = np.zeros((4, 30), np.float32)
    x[:, 3] = 20.0
    torch = torch_cuda()
    xt, one = torch.from_numpy(x).cuda(), f32([1.0] * 4)
    st = ts.ts_token_logp(xt, i32([3] * 4), one, want_stats=True).stats
    g = ts.ts_token_logp_backward(xt, i32([3, 3, 30, -2]), f32([-1.0, math.inf, 1.0, 1.0]), st, one, one, one)
    assert np.isnan(host(g)).all()
    # statistics of a call without tokens serve any of them
    other = ts.ts_token_logp(xt, None, one, want_stats=True).stats
    assert torch.equal(other, st)
    for token in (3, 4):
        check(xt, [token] * 4, [1.0] * 4, [1.0] * 4, None, None, "stats without tokens",
              g=ts.ts_token_logp_backward(xt, i32([token] * 4), one, other, one))


@pytest.mark.parametrize("dtype", TYPES)
def test_same_gradient_bits_whatever_the_batch_and_the_token(dtype):
    # alone, among others, in a batch that passes the caches by, at another address, and with a token that has no gradient
    torch = torch_cuda()
    v, rows = 100003, 720 if dtype != "float32" else 360
    x = make(rows, v, dtype, 50)
    rng = np.random.default_rng(50)
    h, l = rng.standard_normal((2, rows)) * 30
    tokens = rng.integers(0, v, rows)
    tokens[:3] = 5, 50000, v - 1
    none, zero = np.full(rows, -1), np.zeros(rows)
    _, whole = run(x, none, None, zero, h, l)
    _, given = run(x, tokens, None, zero, h, l)
    assert torch.equal(whole, given)
    few = [0, 1, 2, 77, rows - 1]
    for shift in (0, 1):
        y = torch.zeros(len(few) * (v + 5) + shift, dtype=x.dtype, device="cuda")[shift:].view(len(few), v + 5)[:, :v]
        y.copy_(x[few])
        for t in (tokens, none):
            _, g = run(y, t[few], None, zero[few], h[few], l[few])
            assert torch.equal(g, whole[few]), shift
