"""The calls of a decode step together, as a serving loop and a policy update make them: sample, score what was
sampled, report alternatives, take the gradient of a policy loss, evict from the caches."""
import numpy as np
import pytest

import top_select_gumbel_amd as ts
from gpu_helpers import banner, host, torch_cuda
from test_gpu_token_logp import U, tol_log_s

pytestmark = pytest.mark.gpu


def test_decode_loop_with_eviction():
    torch = torch_cuda()
    banner("decode loop: sample, score, evict")
    torch.manual_seed(0)
    batch, heads, dim, vocab, budget = 3, 2, 16, 9000, 24
    rows, slots = batch * heads, budget + 1
    table = torch.randn(vocab, heads * dim, device="cuda")
    k, v = (torch.zeros(batch, heads, slots, dim, device="cuda") for _ in range(2))
    score, position = torch.zeros(rows, slots, device="cuda"), torch.zeros(rows, slots, dtype=torch.int32, device="cuda")
    lengths, keep = torch.zeros(rows, dtype=torch.int32, device="cuda"), torch.full((rows,), budget, dtype=torch.int32, device="cuda")
    temperature = torch.tensor([1.0, 0.7, 0.0], device="cuda")
    tokens = torch.zeros(batch, dtype=torch.int32, device="cuda")
    at_all = torch.arange(slots, device="cuda")
    for step in range(60):
        x = table[tokens.long()].view(batch, heads, dim) + 0.1 * step
        at = lengths.long().view(batch, heads, 1, 1).expand(-1, -1, 1, dim)
        k.scatter_(2, at, x[:, :, None])
        v.scatter_(2, at, x[:, :, None] * 0.5)
        score.scatter_(1, lengths.long()[:, None], 0.0)
        position.scatter_(1, lengths.long()[:, None], step)
        lengths += 1
        logits = (k @ x[..., None])[..., 0] / dim
        logits = logits.view(rows, slots).masked_fill(at_all >= lengths[:, None], -float("inf"))
        w = torch.softmax(logits, 1)
        y = (w.view(batch, heads, 1, slots) @ v).reshape(batch, heads * dim)
        out = (y @ table.t()) / 8
        seed = torch.full((batch,), 1000 + step, dtype=torch.int64, device="cuda")
        tokens, lp, lse, st = ts.ts_sample_rows_logp(out, None, None, temperature, seed)
        r = ts.ts_token_logp(out, tokens, temperature, n_top=4)
        e = ts.ts_cache_evict(score, position, lengths, keep, budget, weights=w.view(rows, 1, slots), k_cache=k, v_cache=v, sinks=1,
                              recent=4, in_place=True)
        torch.cuda.synchronize()
        assert not host(st).any() and not host(r.status).any() and not host(e.status).any()
        # both entry points' tolerances: 3e-6 + 1.2e-7 relative for the sampling one
        a, b = host(lp).astype(float), host(r.logp).astype(float)
        assert (abs(a - b) <= 3e-6 + tol_log_s(vocab) + (1.2e-7 + U) * abs(b)).all(), (a, b)
        assert host(r.rank)[2] == 1 and host(r.logp)[2] == 0.0                     # the greedy row
        assert (host(r.top_idx)[:, 0] == host(out.argmax(1))).all()
        n = host(lengths)
        assert (n == min(step + 1, budget)).all()
        for i in range(rows):
            p = host(position[i])[: n[i]]
            assert len(set(p.tolist())) == n[i] and 0 in p and set(range(max(0, step - 3), step + 1)) <= set(p.tolist())


def test_policy_update_follows_its_gradient():
    """Scores of sampled tokens, an entropy bonus and the gradient, through a linear head: the chain rule's result equals
    autograd's in binary64."""
    torch = torch_cuda()
    banner("policy update")
    torch.manual_seed(1)
    rows, vocab, dim = 24, 8500, 32
    h = torch.randn(rows, dim, device="cuda")
    w = torch.randn(vocab, dim, device="cuda") * 0.3
    x = h @ w.t()
    t = torch.full((rows,), 0.8, device="cuda")
    tokens, _ = ts.ts_sample_rows(x, None, None, t, torch.arange(rows, device="cuda"))
    reward = torch.randn(rows, device="cuda")
    bonus = torch.full((rows,), -0.01, device="cuda")
    f = ts.ts_token_logp(x, tokens, t, want_stats=True)
    g = ts.ts_token_logp_backward(x, tokens, t, f.stats, -reward, bonus)
    y = x.double().requires_grad_(True)
    lp = torch.log_softmax(y / t.double()[:, None], 1)
    loss = (-reward.double() * lp.gather(1, tokens.long()[:, None])[:, 0]).sum() + (bonus.double() * -(lp.exp() * lp).sum(1)).sum()
    want = torch.autograd.grad(loss, y)[0]
    # p <= 1, |d| below 40 here: (|a| + 0.01 * 80) (120 + 3 ln V + 30) u + half a step
    tol = (reward.abs().double()[:, None] + 0.8) / 0.8 * 180 * U
    assert ((g.double() - want).abs() <= tol).all()
    dw = g.t() @ h
    assert torch.isfinite(dw).all() and dw.shape == w.shape
