"""Cases of the token log-probability, its gradient and the cache eviction: inputs, plain forms, 64-bit values.

own = False computes each operator in elementary torch operations; own = True makes the library's calls.

  logp   ts_token_logp: per row of logits the log probability and rank of a given token, the row's entropy and
         log-sum-exp, and the n_top best tokens with their log probabilities
  train  ts_token_logp followed by ts_token_logp_backward: the same, and the gradient of
         sum(grad_logp * logp + grad_entropy * entropy + grad_lse * lse) with respect to the logits
  evict  ts_cache_evict: adds this step's attention weights to each cached position's accumulated weight, keeps the
         `keep` positions of the largest sums (the first `sinks` and the newest `recent` positions before all others)
         and moves kept positions from behind the cut into the freed slots of the key and value caches
"""
import math

import numpy as np
import torch

own = False

TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
LARGEST_LOGITS = 2048 * 151936       # elements of the largest listed train case; drawn cases stay below
LARGEST_CACHE = 32 * 32768           # cached positions of the largest listed evict case


def listed():
    return [
        # one request's next token from a 32000-entry vocabulary: latency alone
        dict(name="logp-one-row", op="logp", rows=1, vocab=32000, type="fp32", n_top=1, masked=0.0, temperature=False),
        # the 64-row decode step of this repository's benchmark, with 20 alternatives to report
        dict(name="logp-decode", op="logp", rows=64, vocab=151936, type="fp32", n_top=20, masked=0.0, temperature=True),
        # a grammar left 0.2% of an odd-sized half-precision vocabulary; rows start at odd addresses
        dict(name="logp-masked-odd", op="logp", rows=33, vocab=50001, type="fp16", n_top=5, masked=0.998, temperature=True),
        # the log probabilities of a batch of whole prompts
        dict(name="logp-prompt", op="logp", rows=1777, vocab=128256, type="bf16", n_top=5, masked=0.0, temperature=False),
        # a toy model's loss, where launches count
        dict(name="train-tiny", op="train", rows=16, vocab=1024, type="fp32", n_top=0, masked=0.0, temperature=False),
        # fp32 logits of an odd vocabulary with padded (masked) entries, tempered policy loss with an entropy bonus
        dict(name="train-odd", op="train", rows=301, vocab=65537, type="fp32", n_top=0, masked=0.01, temperature=True),
        # a 32000-entry vocabulary at a micro-batch of 512 tokens
        dict(name="train-512", op="train", rows=512, vocab=32000, type="bf16", n_top=0, masked=0.0, temperature=False),
        # the largest: a 2048-token micro-batch of the decode vocabulary
        dict(name="train-2048", op="train", rows=2048, vocab=151936, type="bf16", n_top=0, masked=0.0, temperature=True),
        # one short conversation, two heads, odd sizes
        dict(name="evict-short", op="evict", batch=1, heads=2, slots=301, keep=200, queries=3, dim=80, cache="fp16",
             weights="fp32", sinks=1, recent=7, ragged=False, permuted=False),
        # decode step at the cache's budget: each head drops one position of 1025
        dict(name="evict-step", op="evict", batch=8, heads=8, slots=1025, keep=1024, queries=4, dim=128, cache="bf16",
             weights="bf16", sinks=4, recent=64, ragged=False, permuted=True),
        # prompts of different lengths up to 32768 cut to 2048 positions by their last 8 queries of 4 heads each
        dict(name="evict-prompt", op="evict", batch=4, heads=8, slots=32768, keep=2048, queries=32, dim=128, cache="bf16",
             weights="bf16", sinks=4, recent=32, ragged=True, permuted=False),
        # one long document of 131072 positions cut to 8192
        dict(name="evict-long", op="evict", batch=1, heads=8, slots=131072, keep=8192, queries=4, dim=128, cache="bf16",
             weights="fp32", sinks=4, recent=256, ragged=False, permuted=False),
    ]


def _log_uniform(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["logp", "train", "evict"])
    if op == "evict":
        heads = rng.choice([1, 2, 3, 4, 8])
        batch = _log_uniform(rng, 1, 16)
        slots = _log_uniform(rng, 17, min(131072, max(64, LARGEST_CACHE // (heads * batch))))
        keep = max(1, int(slots * rng.uniform(0.05, 1.0)))
        # rows x queries x slots weights: no more than the largest listed case's
        queries = _log_uniform(rng, 1, max(1, min(64, 32 * LARGEST_CACHE // (heads * batch * slots))))
        return dict(op=op, batch=batch, heads=heads, slots=slots, keep=keep, queries=queries,
                    dim=rng.choice([33, 64, 80, 96, 128]), cache=rng.choice(list(TYPES)), weights=rng.choice(list(TYPES)),
                    sinks=rng.choice([0, 1, 4]), recent=rng.randrange(0, 65), ragged=rng.random() < 0.5,
                    permuted=rng.random() < 0.5)
    vocab = _log_uniform(rng, 100, 262144)
    rows = _log_uniform(rng, 1, max(1, min(4096, LARGEST_LOGITS // (2 * vocab))))
    return dict(op=op, rows=rows, vocab=vocab, type=rng.choice(list(TYPES)),
                n_top=0 if op == "train" else rng.choice([0, 1, 5, 20, 64]), masked=rng.choice([0.0, 0.0, 0.01, 0.5, 0.99]),
                temperature=rng.random() < 0.5)


# ---------------------------------------------------------------- inputs
def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed * 1000003 + 17)
    if case["op"] == "evict":
        return _prepare_evict(case, gen, dev)
    rows, vocab = case["rows"], case["vocab"]
    x = torch.randn((rows, vocab), generator=gen, device=dev).mul_(2.5)
    # 20 likely tokens a row, as the decode workload has them
    head = torch.randint(0, vocab, (rows, 20), generator=gen, device=dev)
    x.scatter_add_(1, head, torch.full((rows, 20), 8.0, device=dev))
    best = x.argmax(1, keepdim=True)
    if case["masked"]:
        keep = torch.rand((rows, vocab), generator=gen, device=dev) >= case["masked"]
        keep.scatter_(1, best, True)
        x.masked_fill_(~keep, -math.inf)
        del keep
    x = x.to(TYPES[case["type"]])
    # the given tokens: the best one, one of the likely ones, any one; one row in sixteen has none
    pick = torch.randint(0, 16, (rows,), generator=gen, device=dev)
    tokens = torch.where(pick < 6, best[:, 0], torch.where(pick < 11, head[:, 0],
                         torch.randint(0, vocab, (rows,), generator=gen, device=dev)))
    tokens = torch.where(pick == 15, torch.full_like(tokens, -1), tokens).to(torch.int32)
    state = dict(case=case, x=x, tokens=tokens, temperature=None)
    if case["temperature"]:
        state["temperature"] = torch.rand(rows, generator=gen, device=dev).add_(0.5)
    if case["op"] == "train":
        state["g_logp"] = torch.randn(rows, generator=gen, device=dev)
        state["g_entropy"] = torch.randn(rows, generator=gen, device=dev).mul_(0.01)
        state["g_lse"] = torch.randn(rows, generator=gen, device=dev).mul_(0.001)
    return state


def _prepare_evict(case, gen, dev):
    rows, slots = case["batch"] * case["heads"], case["slots"]
    lengths = torch.full((rows,), slots, dtype=torch.int32, device=dev)
    if case["ragged"]:   # all heads of a sequence have its length
        u = torch.rand((case["batch"], 1), generator=gen, device=dev)
        lengths = (1 + u * (slots - 1)).to(torch.int32).expand(-1, case["heads"]).reshape(-1).contiguous()
    at = torch.arange(slots, device=dev)
    live = at[None, :] < lengths[:, None]
    # accumulated weights are heavy-tailed; many positions hold exactly nothing
    score = torch.exp(torch.randn((rows, slots), generator=gen, device=dev) * 2.0 - 4.0)
    score[torch.rand((rows, slots), generator=gen, device=dev) < 0.2] = 0.0
    logits = torch.randn((rows, case["queries"], slots), generator=gen, device=dev).mul_(2.5)
    logits.masked_fill_(~live[:, None, :], -math.inf)
    weights = torch.softmax(logits, -1).to(TYPES[case["weights"]])
    if case["permuted"]:   # slots that earlier evictions have filled out of order
        order = torch.rand((rows, slots), generator=gen, device=dev).masked_fill_(~live, 2.0).argsort(1)
        position = torch.empty((rows, slots), dtype=torch.int64, device=dev)
        position.scatter_(1, order, at.expand(rows, -1).contiguous())
    else:
        position = at.expand(rows, -1)
    position = torch.where(live, position, torch.full_like(position, -1)).to(torch.int32).contiguous()
    shape = (case["batch"], case["heads"], slots, case["dim"])
    cache = TYPES[case["cache"]]
    return dict(case=case, score=score, weights=weights, position=position, lengths=lengths,
                keep=torch.full((rows,), case["keep"], dtype=torch.int32, device=dev),
                k=torch.randn(shape, generator=gen, device=dev).to(cache), v=torch.randn(shape, generator=gen, device=dev).to(cache))


# ---------------------------------------------------------------- one pass
def run(state):
    op = state["case"]["op"]
    if op == "evict":
        return _evict_own(state) if own else _evict_plain(state)
    if op == "train":
        return _train_own(state) if own else _train_plain(state)
    return _logp_own(state) if own else _logp_plain(state)


def _logp_own(s):
    import top_select_gumbel_amd as ts
    r = ts.ts_token_logp(s["x"], s["tokens"], s["temperature"], n_top=s["case"]["n_top"])
    return dict(logp=r.logp, rank=r.rank, entropy=r.entropy, lse=r.lse, top_idx=r.top_idx, top_logp=r.top_logp, status=r.status)


def _train_own(s):
    import top_select_gumbel_amd as ts
    r = ts.ts_token_logp(s["x"], s["tokens"], s["temperature"], want_rank=False, want_stats=True)
    grad = ts.ts_token_logp_backward(s["x"], s["tokens"], s["temperature"], r.stats, s["g_logp"], s["g_entropy"], s["g_lse"])
    return dict(logp=r.logp, entropy=r.entropy, lse=r.lse, grad=grad, status=r.status)


def _evict_own(s):
    import top_select_gumbel_amd as ts
    c = s["case"]
    r = ts.ts_cache_evict(s["score"], s["position"], s["lengths"], s["keep"], c["keep"], weights=s["weights"],
                          k_cache=s["k"], v_cache=s["v"], sinks=c["sinks"], recent=c["recent"])
    return dict(source=r.source, lengths=r.lengths, score=r.score, position=r.position, status=r.status, k=s["k"], v=s["v"])


def _distribution(s):
    """Plain: the tempered logits less their maximum, log S and the log-sum-exp of every row, in 32 bits."""
    z = s["x"].float()
    if s["temperature"] is not None:
        z = z / s["temperature"][:, None]
    m = z.amax(1, keepdim=True)
    d = z - m
    e = torch.exp(d)
    total = e.sum(1, dtype=torch.float64)
    log_s = torch.log(total)
    return d, e, total, log_s, m[:, 0].double() + log_s


def _statistics(s):
    d, e, total, log_s, lse = _distribution(s)
    entropy = log_s - torch.where(e > 0, e * d, torch.zeros_like(d)).sum(1, dtype=torch.float64) / total
    none = s["tokens"] < 0
    at = s["tokens"].long().clamp(min=0)[:, None]
    logp = torch.where(none, torch.zeros_like(log_s), d.gather(1, at)[:, 0].double() - log_s)
    return d, e, total, log_s, lse, entropy, none, at, logp


def _logp_plain(s):
    n = s["case"]["n_top"]
    x = s["x"]
    d, e, total, log_s, lse, entropy, none, at, logp = _statistics(s)
    xt = x.gather(1, at)
    ids = torch.arange(x.shape[1], device=x.device)
    rank = 1 + ((x > xt) | ((x == xt) & (ids < at))).sum(1)
    rank = torch.where(none, torch.zeros_like(rank), rank).to(torch.int32)
    # value descending, then id ascending: one whole number orders both (-0 counts as +0)
    bits = (x.float() + 0.0).view(torch.int32).long()
    key = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits)
    key = (key << 31) + (0x7FFFFFFF - ids)
    top = torch.topk(key, min(n, x.shape[1]), dim=1).indices
    top_logp = (d.gather(1, top).double() - log_s[:, None]).float()
    top = torch.where(x.gather(1, top) > -math.inf, top, torch.full_like(top, -1)).to(torch.int32)
    more = n - top.shape[1]
    if more:
        top = torch.nn.functional.pad(top, (0, more), value=-1)
        top_logp = torch.nn.functional.pad(top_logp, (0, more), value=-math.inf)
    return dict(logp=logp.float(), rank=rank, entropy=entropy.float(), lse=lse.float(), top_idx=top if n else None,
                top_logp=top_logp if n else None, status=torch.zeros_like(rank))


def _train_plain(s):
    d, e, total, log_s, lse, entropy, none, at, logp = _statistics(s)
    p = e / total.float()[:, None]
    lp = torch.where(e > 0, d - log_s.float()[:, None], torch.zeros_like(d))
    a = torch.where(none, torch.zeros_like(s["g_logp"]), s["g_logp"])
    g = p * ((s["g_lse"] - a)[:, None] - s["g_entropy"][:, None] * (lp + entropy.float()[:, None]))
    g.scatter_add_(1, at, a[:, None])
    if s["temperature"] is not None:
        g = g / s["temperature"][:, None]
    return dict(logp=logp.float(), entropy=entropy.float(), lse=lse.float(), grad=g.to(s["x"].dtype),
                status=torch.zeros_like(s["tokens"]))


def _evict_plain(s):
    c = s["case"]
    score, position = s["score"], s["position"]
    rows, slots = score.shape
    width = c["keep"]
    at = torch.arange(slots, device=score.device)
    live = at < s["lengths"][:, None]
    # sums in 64 bits, rounded once: the order of two near ones decides what stays
    total = (score.double() + s["weights"].double().sum(1)).float()
    newest = torch.where(live, position, torch.full_like(position, -1)).amax(1, keepdim=True)
    first = (position < c["sinks"]) | (position > newest - c["recent"])
    bits = (total + 0.0).view(torch.int32).long()
    key = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits) + (1 << 31)
    key = torch.where(live, key + (first.long() << 32) + 1, torch.zeros_like(key))
    order = torch.argsort(key, dim=1, descending=True, stable=True)
    rank = torch.empty_like(order).scatter_(1, order, at.expand(rows, -1).contiguous())
    n = torch.minimum(s["keep"], s["lengths"])[:, None].long()
    kept = rank < n
    hole, filler = (at < n) & ~kept, (at >= n) & kept
    # the i-th freed slot takes the i-th kept position from behind the cut
    fillers = torch.full((rows, slots + 1), -1, dtype=torch.int64, device=score.device)
    fillers.scatter_(1, torch.where(filler, filler.cumsum(1) - 1, torch.full_like(order, slots)), at.expand(rows, -1).contiguous())
    source = torch.where(hole, fillers.gather(1, (hole.cumsum(1) - 1).clamp(min=0)), at.expand(rows, -1))[:, :width]
    inside = at[:width] < n
    new_score = torch.where(inside, total.gather(1, source), torch.zeros_like(total[:, :width]))
    new_position = torch.where(inside, position.gather(1, source), torch.full_like(position[:, :width], -1))
    from_slot = source.view(c["batch"], c["heads"], width, 1).expand(-1, -1, -1, c["dim"])
    s["k"][:, :, :width] = s["k"].gather(2, from_slot)
    s["v"][:, :, :width] = s["v"].gather(2, from_slot)
    return dict(source=torch.where(inside, source, torch.full_like(source, -1)).to(torch.int32), lengths=n[:, 0].to(torch.int32),
                score=new_score, position=new_position, status=torch.zeros_like(s["lengths"]), k=s["k"], v=s["v"])


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    if case["op"] == "evict":
        rows, slots, keep = case["batch"] * case["heads"], case["slots"], case["keep"]
        size = {"fp32": 4, "bf16": 2, "fp16": 2}
        # of the kept positions, the share that lies behind the cut has to move
        moved = keep * (1.0 - keep / slots)
        reads = slots * (4 + 4 + case["queries"] * size[case["weights"]]) + 2 * moved * case["dim"] * size[case["cache"]]
        writes = keep * (4 + 4 + 4) + 2 * moved * case["dim"] * size[case["cache"]]
        share = 0.5 if case["ragged"] else 1.0
        return {"bytes": rows * share * (reads + writes), "flops": rows * share * slots * (case["queries"] + 1)}
    n = case["rows"] * case["vocab"]
    size = TYPES[case["type"]].itemsize
    if case["op"] == "train":
        return {"bytes": n * size * 2 + case["rows"] * 32, "flops": n * 12}
    return {"bytes": n * size + case["rows"] * (24 + 8 * case["n_top"]), "flops": n * 6}


# ---------------------------------------------------------------- 64-bit values
def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "evict":
        return _exact_evict(state)
    parts = []
    rows = max(1, (1 << 27) // case["vocab"])   # a slab of rows at a time: 1 GB of doubles
    for r in range(0, case["rows"], rows):
        parts.append(_exact_rows(state, slice(r, r + rows)))
    return {k: None if parts[0][k] is None else torch.cat([p[k] for p in parts]) for k in parts[0]}


def _exact_rows(s, rows):
    x = s["x"][rows].double()
    t = 1.0 if s["temperature"] is None else s["temperature"][rows].double()[:, None]
    train = s["case"]["op"] == "train"
    masked = x == -math.inf
    x.requires_grad_(train)
    with torch.set_grad_enabled(train):
        z = x / t
        lse = torch.logsumexp(z, 1)
        lp = z - lse[:, None]
        p = torch.exp(lp)
        entropy = -(p * lp.masked_fill(masked, 0.0)).sum(1)
        token = s["tokens"][rows].long()
        given = token >= 0
        logp = torch.where(given, lp.gather(1, token.clamp(min=0)[:, None])[:, 0], torch.zeros_like(lse))
        if train:
            loss = (s["g_logp"][rows].double() * torch.where(given, logp, torch.zeros_like(logp)).masked_fill(~given, 0.0)
                    + s["g_entropy"][rows].double() * entropy + s["g_lse"][rows].double() * lse)
            grad = torch.autograd.grad(loss.sum(), x)[0]
    out = dict(logp=logp.detach(), entropy=entropy.detach(), lse=lse.detach(), status=None)
    if train:
        return dict(out, grad=grad)
    n = s["case"]["n_top"]
    top = None
    if n:   # the values alone: whichever of two equal ones comes first, they are the same
        top = torch.topk(lp, min(n, lp.shape[1]), dim=1).values
        top = torch.nn.functional.pad(top, (0, n - top.shape[1]), value=-math.inf)
    return dict(out, rank=None, top_idx=None, top_logp=top)


def _exact_evict(s):
    c = s["case"]
    rows, slots = s["score"].shape
    score = s["score"].double().cpu().numpy()
    # by the definition the sums are kept in fp32, and what is kept goes by those
    total = np.empty_like(score)
    for r in range(rows):
        total[r] = score[r] + s["weights"][r].double().cpu().numpy().sum(0)
    held = total.astype(np.float32)
    position, lengths = s["position"].cpu().numpy(), s["lengths"].cpu().numpy()
    out_score = np.zeros((rows, c["keep"]))
    k, v = s["k"], s["v"]
    for r in range(rows):
        n = int(lengths[r])
        pos = position[r, :n]
        first = (pos < c["sinks"]) | (pos > pos.max() - c["recent"])
        order = np.lexsort((np.arange(n), -held[r, :n], ~first))
        m = min(c["keep"], n)
        stay = np.sort(order[:m])
        source = np.arange(m)
        source[np.setdiff1d(np.arange(m), stay)] = stay[stay >= m]
        out_score[r, :m] = total[r, source]
        b, h = divmod(r, c["heads"])
        at = torch.from_numpy(source).to(k.device)
        k[b, h, :m] = k[b, h][at]
        v[b, h, :m] = v[b, h][at]
    return dict(source=None, lengths=None, score=torch.from_numpy(out_score), position=None, status=None, k=k, v=v)
