"""Cases of attention over a paged key / value cache and of the cache's pages: inputs, plain forms, 64-bit values.

own = False computes each operator in elementary torch operations; own = True makes the library's calls.

A cache holds pages [pages, kv_heads, page_slots, dim]; position j of sequence b lies in page table[b, j // page_slots],
slot j % page_slots. refs counts the sequences that hold a page; a page with count 0 is free.

  attend   ts_cache_attend: one new token's queries over each sequence's cached positions, with the log-sum-exp and, for
           eviction by attention weight, the weights themselves
  append   ts_cache_append: the keys and values of each sequence's newest tokens into their pages
  fork     ts_pages_fork: every sequence of the next step continues one of this step's, grown by n_new positions: whole pages
           are shared, a part-filled last page is copied for every child but the first, pages that nobody holds any
           longer are free, and fresh ones are the lowest free ones in order
  compact  ts_pages_compact: moves the pages in use to the lowest numbers and renumbers the tables
  copy     ts_pages_copy: whole pages from one number to another, in every layer's pool
"""
import math

import numpy as np
import torch

own = False

TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
LARGEST_CACHE = 2 * 8 * 131072 * 128       # elements of the keys of the largest listed attend case; drawn cases stay below
LARGEST_MOVED = 1024 * 8 * 16384           # elements that the largest listed copy case moves
NO_PAGE = 10                               # TS_ROW_NO_PAGE


def listed():
    return [
        # one short conversation in fp32, odd sizes: latency alone
        dict(name="attend-one", op="attend", batch=1, kv_heads=2, group=2, dim=80, type="fp32", length=301, page=24,
             ragged=False, window=0, weights=""),
        # a 64-row decode step: conversations of any length up to 4096
        dict(name="attend-step", op="attend", batch=64, kv_heads=8, group=4, dim=128, type="bf16", length=4096, page=16,
             ragged=True, window=0, weights=""),
        # a decode step whose weights go to the eviction of one position of 1025: a dense cache, one page a sequence
        dict(name="attend-evict", op="attend", batch=8, kv_heads=8, group=4, dim=128, type="bf16", length=1025, page=1025,
             ragged=False, window=0, weights="bf16"),
        # two long documents: few rows, split over the length
        dict(name="attend-long", op="attend", batch=2, kv_heads=8, group=8, dim=128, type="fp16", length=131072, page=64,
             ragged=False, window=0, weights=""),
        # one new token of each of 64 conversations
        dict(name="append-step", op="append", batch=64, kv_heads=8, dim=128, type="bf16", length=1000, page=16, new=1),
        # prompts of several lengths up to 16384
        dict(name="append-prompt", op="append", batch=5, kv_heads=8, dim=128, type="fp16", length=16384, page=64, new=16384),
        # bookkeeping of a decode step: 64 conversations grow by a token, some ended and others start
        dict(name="fork-step", op="fork", seqs=64, children=64, length=4000, page=16, pages=20000, shared=8, new=1, beams=False,
             ended=0.05, pools=8, heads=2, dim=64, type="bf16"),
        # beam search: 64 beams go on from some of the last step's
        dict(name="fork-beams", op="fork", seqs=64, children=64, length=700, page=16, pages=4096, shared=16, new=1, beams=True,
             ended=0.0, pools=16, heads=8, dim=128, type="bf16"),
        # a toy cache of odd sizes, a third in use
        dict(name="compact-small", op="compact", seqs=5, length=60, page=12, pages=75, used=0.33, pools=2, heads=3, dim=33, type="fp16"),
        # a cache of 8192 pages, half in use and scattered after a long time of serving
        dict(name="compact-large", op="compact", seqs=48, length=1500, page=16, pages=8192, used=0.55, pools=8, heads=8, dim=128,
             type="bf16"),
        # three pages of two layers, odd sizes
        dict(name="copy-three", op="copy", pairs=3, page=12, pages=40, pools=4, heads=3, dim=33, type="fp32"),
        # a preempted batch's 1024 pages of four layers into another part of the cache
        dict(name="copy-batch", op="copy", pairs=1024, page=16, pages=4096, pools=8, heads=8, dim=128, type="bf16"),
    ]


def _log_uniform(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "append", "fork", "compact", "copy"])
    dim = rng.choice([33, 64, 80, 96, 128, 256])
    kind = rng.choice(list(TYPES))
    page = rng.choice([1, 8, 16, 16, 24, 32, 64, 257])
    if op == "attend":
        kv_heads = rng.choice([1, 2, 4, 8])
        group = rng.choice([1, 2, 4, 7, 8, 16, 32])
        batch = _log_uniform(rng, 1, 200)
        # keys of at most a quarter of the largest case's elements; the plain form's scores, for every query head, too
        length = _log_uniform(rng, 1, max(2, min(131072, LARGEST_CACHE // (4 * batch * kv_heads * max(dim, 4 * group)))))
        return dict(op=op, batch=batch, kv_heads=kv_heads, group=group, dim=dim, type=kind, length=length, page=page,
                    ragged=rng.random() < 0.6, window=rng.choice([0, 0, 1, 128, 1000]), weights=rng.choice(["", "", "fp32", "bf16", "fp16"]))
    if op == "append":
        kv_heads = rng.choice([1, 2, 3, 8])
        batch = _log_uniform(rng, 1, 300)
        length = _log_uniform(rng, 1, max(2, min(16384, LARGEST_CACHE // (16 * batch * kv_heads * dim))))
        return dict(op=op, batch=batch, kv_heads=kv_heads, dim=dim, type=kind, length=length, page=page,
                    new=rng.choice([1, 1, 5, length]))
    heads = rng.choice([1, 2, 3, 8])
    pools = rng.choice([1, 2, 4, 8, 40])
    size = page * heads * dim
    if op == "copy":
        pages = _log_uniform(rng, 2, max(3, min(20000, 2 * LARGEST_MOVED // (size * pools))))
        return dict(op=op, pairs=rng.randint(1, pages // 2), page=page, pages=pages, pools=pools, heads=heads, dim=dim, type=kind)
    pages = _log_uniform(rng, 40, max(50, min(60000, 2 * LARGEST_MOVED // (size * pools))))
    if op == "compact":
        seqs = _log_uniform(rng, 1, min(200, pages // 4))
        used = rng.uniform(0.05, 0.95)
        return dict(op=op, seqs=seqs, length=max(1, int(used * pages / seqs * page)), page=page, pages=pages, used=used, pools=pools,
                    heads=heads, dim=dim, type=kind)
    seqs = _log_uniform(rng, 1, min(200, pages // 8))
    shared = rng.choice([0, 0, 2])
    return dict(op=op, seqs=seqs, children=max(1, int(seqs * rng.uniform(0.5, 1.5))), page=page, pages=pages, shared=shared,
                length=max((shared + 1) * page, int(rng.uniform(0.1, 0.9) * pages / seqs * page)), new=rng.choice([0, 1, 1, 40]),
                beams=rng.random() < 0.5, ended=rng.choice([0.0, 0.1, 0.5]), pools=pools, heads=heads, dim=dim, type=kind)


# ---------------------------------------------------------------- inputs
def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed * 1000003 + 29)
    return {"attend": _prepare_attend, "append": _prepare_append, "fork": _prepare_fork, "compact": _prepare_compact,
            "copy": _prepare_copy}[case["op"]](case, gen, dev)


def _normal(shape, kind, gen, dev):
    return torch.randn(shape, generator=gen, device=dev).to(TYPES[kind])


def _tables(lengths, page, width, pages, gen, dev):
    """Page numbers in no order, as a cache that has run for long has them; -1 past a sequence's end."""
    order = torch.randperm(pages, generator=gen, device=dev)[: lengths.numel() * width].view(-1, width)
    held = torch.arange(width, device=dev)[None, :] < ((lengths + page - 1) // page)[:, None]
    return torch.where(held, order, torch.full_like(order, -1)).to(torch.int32)


def _prepare_attend(c, gen, dev):
    b, n, page = c["batch"], c["length"], c["page"]
    lengths = torch.full((b,), n, dtype=torch.int32, device=dev)
    if c["ragged"]:
        u = torch.rand(b, generator=gen, device=dev)
        lengths = (1 + u * (n - 1)).to(torch.int32)
    width = (n + page - 1) // page
    pages = b * width + (0 if width == 1 else 7)
    table = _tables(lengths, page, width, pages, gen, dev)
    if width == 1:
        table = torch.arange(b, dtype=torch.int32, device=dev).view(b, 1)
    shape = (pages, c["kv_heads"], page, c["dim"])
    # queries along a few keys' direction: some positions take most of the weight, as in earnest
    k = _normal(shape, c["type"], gen, dev)
    q = torch.randn((b, c["kv_heads"] * c["group"], c["dim"]), generator=gen, device=dev).mul_(1.7).to(TYPES[c["type"]])
    return dict(case=c, q=q, k=k, v=_normal(shape, c["type"], gen, dev), table=table, lengths=lengths)


def _prepare_append(c, gen, dev):
    b, page = c["batch"], c["page"]
    u = torch.rand(b, generator=gen, device=dev)
    if c["new"] == 1:
        lengths = (1 + u * (c["length"] - 1)).to(torch.int32)
        new = torch.ones_like(lengths)
    else:
        lengths = torch.clamp((u * c["length"]).to(torch.int32) + 1, max=c["length"])
        new = torch.clamp(lengths, max=c["new"])
    offsets = torch.zeros(b + 1, dtype=torch.int32, device=dev)
    offsets[1:] = new.cumsum(0)
    width = (c["length"] + page - 1) // page
    pages = b * width + 3
    shape = (pages, c["kv_heads"], page, c["dim"])
    tokens = int(offsets[-1])
    return dict(case=c, k=_normal(shape, c["type"], gen, dev), v=_normal(shape, c["type"], gen, dev),
                k_new=_normal((tokens, c["kv_heads"], c["dim"]), c["type"], gen, dev),
                v_new=_normal((tokens, c["kv_heads"], c["dim"]), c["type"], gen, dev),
                offsets=offsets, lengths=lengths, table=_tables(lengths, page, width, pages, gen, dev))


def _pools(c, gen, dev):
    """The pools, and what a program that makes the library's calls keeps beside them: their addresses, taken once."""
    pools = [_normal((c["pages"], c["heads"], c["page"], c["dim"]), c["type"], gen, dev) for _ in range(c["pools"])]
    plan = None
    if own:
        import top_select_gumbel_amd as ts
        plan = ts.PagePools(pools)
    return dict(pools=pools, plan=plan)


def _sequences(c, seqs, shared, gen, dev):
    """Tables of sequences of random lengths that hold the first `shared` pages together; and the pages' counts."""
    page = c["page"]
    low = shared * page
    u = torch.rand(seqs, generator=gen, device=dev)
    lengths = (low + 1 + u * (c["length"] - low - 1)).to(torch.int32)
    # room in the table for what may be added
    width = (c["length"] + c.get("new", 0) + page - 1) // page
    held = (lengths.long() + page - 1) // page
    at = torch.arange(width, device=dev)
    inside = at < held[:, None]
    own_page = inside & (at >= shared)
    # as many pages as there are, in no order: the shared ones first, then each sequence's own
    order = torch.randperm(c["pages"], generator=gen, device=dev)
    rank = own_page.reshape(-1).long().cumsum(0).view(seqs, width) - 1 + shared
    table = torch.where(own_page, order[rank.clamp(max=c["pages"] - 1)], order[at.clamp(max=c["pages"] - 1)][None, :])
    # where the pages are used up, a sequence ends
    short = (own_page & (rank >= c["pages"])).any(1)
    lengths = torch.where(short, torch.zeros_like(lengths), lengths)
    table = torch.where(inside & ~short[:, None], table, torch.full_like(table, -1))
    refs = torch.zeros(c["pages"], dtype=torch.int32, device=dev)
    refs.scatter_add_(0, table.clamp(min=0).reshape(-1), (table >= 0).reshape(-1).to(torch.int32))
    return table.to(torch.int32), lengths, refs


def _prepare_fork(c, gen, dev):
    table, lengths, refs = _sequences(c, c["seqs"], c["shared"], gen, dev)
    n = c["children"]
    if c["beams"]:
        parent = torch.randint(0, c["seqs"], (n,), generator=gen, device=dev)
    else:
        parent = torch.arange(n, device=dev)
        parent = torch.where(parent < c["seqs"], parent, torch.full_like(parent, -1))
    gone = torch.rand(n, generator=gen, device=dev) < c["ended"]
    parent = torch.where(gone, torch.full_like(parent, -1), parent).to(torch.int32)
    new = torch.full((n,), c["new"], dtype=torch.int32, device=dev)
    return dict(case=c, table=table, lengths=lengths, refs=refs, parent=parent, n_new=new, **_pools(c, gen, dev))


def _prepare_compact(c, gen, dev):
    table, lengths, refs = _sequences(c, c["seqs"], 0, gen, dev)
    return dict(case=c, table=table, lengths=lengths, refs=refs, **_pools(c, gen, dev))


def _prepare_copy(c, gen, dev):
    order = torch.randperm(c["pages"], generator=gen, device=dev).to(torch.int32)
    return dict(case=c, source=order[: c["pairs"]].contiguous(), target=order[c["pairs"]: 2 * c["pairs"]].contiguous(),
                **_pools(c, gen, dev))


# ---------------------------------------------------------------- one pass
def run(state):
    name = "_%s_%s" % (state["case"]["op"], "own" if own else "plain")
    return globals()[name](state)


def _attend_own(s):
    import top_select_gumbel_amd as ts
    c = s["case"]
    kind = TYPES[c["weights"]] if c["weights"] else None
    r = ts.ts_cache_attend(s["q"], s["k"], s["v"], s["table"], s["lengths"], window=c["window"],
                           weights_slots=c["length"] if c["weights"] else 0, weights_dtype=kind)
    return dict(out=r.out, lse=r.lse, weights=r.weights, status=r.status)


def _append_own(s):
    import top_select_gumbel_amd as ts
    status = ts.ts_cache_append(s["k_new"], s["v_new"], s["offsets"], s["k"], s["v"], s["table"], s["lengths"])
    return dict(k=s["k"], v=s["v"], status=status)


def _fork_own(s):
    import top_select_gumbel_amd as ts
    r = ts.ts_pages_fork(s["table"], s["lengths"], s["refs"], s["parent"], s["case"]["page"], n_new=s["n_new"], pools=s["plan"])
    return dict(table=r.table, lengths=r.lengths, refs=r.refs, status=r.status, pools=s["pools"])


def _compact_own(s):
    import top_select_gumbel_amd as ts
    r = ts.ts_pages_compact(s["table"], s["lengths"], s["refs"], s["case"]["page"], pools=s["plan"])
    return dict(table=r.table, refs=r.refs, map=r.map, count=r.count, status=r.status, pools=s["pools"])


def _copy_own(s):
    import top_select_gumbel_amd as ts
    return dict(status=ts.ts_pages_copy(s["source"], s["target"], s["plan"]), pools=s["pools"])


def _attend_plain(s):
    c = s["case"]
    b, hk, g, dim, page = c["batch"], c["kv_heads"], c["group"], c["dim"], c["page"]
    width = s["table"].shape[1]
    pages = s["table"].long().clamp(min=0)
    at = torch.arange(width * page, device=pages.device)
    n = s["lengths"].long()[:, None]
    attended = at < n
    if c["window"]:
        attended = attended & (at >= n - c["window"])

    def dense(x):   # [b, kv_heads, positions, dim] in 32 bits
        return x[pages].transpose(1, 2).reshape(b, hk, width * page, dim).float()
    q = s["q"].float().view(b, hk, g, dim).transpose(2, 3).contiguous()
    scores = torch.matmul(dense(s["k"]), q).mul_(dim ** -0.5)
    scores = scores.masked_fill_(~attended[:, None, :, None], -math.inf)
    top = scores.amax(2, keepdim=True)
    p = torch.exp(scores - top)
    total = p.sum(2, keepdim=True)
    p = (p / total).transpose(2, 3).contiguous()
    v = dense(s["v"]).masked_fill_(~attended[:, None, :, None], 0.0)
    out = torch.matmul(p, v).reshape(b, hk * g, dim).to(s["q"].dtype)
    lse = (top + torch.log(total)).reshape(b, hk * g)
    weights = None
    if c["weights"]:
        weights = p.reshape(b, hk * g, width * page)[:, :, : c["length"]].to(TYPES[c["weights"]])
    return dict(out=out, lse=lse, weights=weights, status=torch.zeros_like(s["lengths"]))


def _append_plain(s):
    page = s["case"]["page"]
    offsets = s["offsets"].long()
    token = torch.arange(s["k_new"].shape[0], device=offsets.device)
    seq = torch.searchsorted(offsets, token, right=True) - 1
    position = s["lengths"].long()[seq] - (offsets[seq + 1] - token)
    where = s["table"].long()[seq, position // page]
    slot = position % page
    s["k"][where, :, slot] = s["k_new"]
    s["v"][where, :, slot] = s["v_new"]
    return dict(k=s["k"], v=s["v"], status=torch.zeros_like(s["lengths"]))


def _fork_plain(s):
    page = s["case"]["page"]
    table, lengths, parent, new = s["table"].long(), s["lengths"].long(), s["parent"].long(), s["n_new"].long()
    (seqs, width), n = table.shape, parent.numel()
    at = torch.arange(width, device=table.device)
    child = torch.arange(n, device=table.device)
    has, of = parent >= 0, parent.clamp(min=0)
    count = torch.zeros(seqs, dtype=torch.int64, device=table.device).scatter_add_(0, of, has.long())
    first = torch.full((seqs,), n, dtype=torch.int64, device=table.device)
    first.scatter_reduce_(0, of, torch.where(has, child, torch.full_like(child, n)), "amin")
    whole = (lengths // page)[:, None]
    part = (lengths % page > 0)[:, None] & (at == whole)
    change = torch.where(at < whole, (count - 1)[:, None], torch.where(part & (count == 0)[:, None], -1, 0))
    refs = s["refs"].long().scatter_add(0, table.clamp(min=0).reshape(-1), change.reshape(-1))
    free = refs <= 0
    order = torch.argsort((~free).to(torch.int8), stable=True)
    old = torch.where(has, lengths[of], torch.zeros_like(new))
    copies = has & (first[of] != child) & (old % page > 0)
    before, after = (old + page - 1) // page, (old + new + page - 1) // page
    need = copies.long() + after - before
    start = need.cumsum(0) - need
    fits = start + need <= free.sum()
    empty = ~fits & copies
    out_lengths = torch.where(fits, old + new, torch.where(empty, 0, old))
    # a child that is left empty gives back what it would have shared
    back = (empty[:, None] & (at < (old // page)[:, None])).long()
    refs.scatter_add_(0, table[of].clamp(min=0).reshape(-1), -back.reshape(-1))
    out = torch.where((at < before[:, None]) & ~empty[:, None], table[of], -1)
    fresh = torch.where(copies[:, None] & (at == (old // page)[:, None]), 0,
                        torch.where((at >= before[:, None]) & (at < after[:, None]), copies.long()[:, None] + at - before[:, None], -1))
    fresh = torch.where(fits[:, None] & (fresh >= 0), fresh + start[:, None], -1)
    number = order[fresh.clamp(min=0, max=order.numel() - 1)]
    out = torch.where(fresh >= 0, number, out)
    refs[number[fresh >= 0]] = 1
    moved = (fits & copies).nonzero()[:, 0]
    last = (old // page)[moved]
    for pool in s["pools"]:
        pool[out[moved, last]] = pool[table[of[moved], last]]
    return dict(table=out.to(torch.int32), lengths=out_lengths.to(torch.int32), refs=refs.to(torch.int32),
                status=torch.where(fits, 0, NO_PAGE).to(torch.int32), pools=s["pools"])


def _compact_plain(s):
    refs = s["refs"]
    at = torch.arange(refs.numel(), device=refs.device)
    live = refs > 0
    n = live.sum()
    hole, mover = (~live & (at < n)).nonzero()[:, 0], (live & (at >= n)).nonzero()[:, 0]
    to = torch.where(live, at, -1)
    to[mover] = hole
    out_refs = torch.where(live & (at < n), refs, 0)
    out_refs[hole] = refs[mover]
    table = torch.where(s["table"] >= 0, to[s["table"].long().clamp(min=0)], -1)
    for pool in s["pools"]:
        pool[hole] = pool[mover]
    return dict(table=table.to(torch.int32), refs=out_refs, map=to.to(torch.int32), count=n.to(torch.int32).view(1),
                status=torch.zeros_like(s["lengths"]), pools=s["pools"])


def _copy_plain(s):
    for pool in s["pools"]:
        pool[s["target"].long()] = pool[s["source"].long()]
    return dict(status=torch.zeros_like(s["source"]), pools=s["pools"])


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    op, size, dim = case["op"], TYPES[case["type"]].itemsize, case["dim"]
    if op == "attend":
        heads = case["kv_heads"] * case["group"]
        mean = case["length"] / 2 if case["ragged"] else case["length"]
        seen = min(mean, case["window"]) if case["window"] else mean
        cached = case["batch"] * seen
        b = 2 * cached * case["kv_heads"] * dim * size + cached / case["page"] * 4 + case["batch"] * heads * (2 * dim * size + 4)
        if case["weights"]:
            b += case["batch"] * heads * case["length"] * TYPES[case["weights"]].itemsize
        return {"bytes": b, "flops": 4 * cached * heads * dim}
    if op == "append":
        tokens = case["batch"] * (1 if case["new"] == 1 else min(case["new"], case["length"] / 2))
        return {"bytes": 4 * tokens * case["kv_heads"] * dim * size + tokens * 4, "flops": 0}
    page_bytes = case["page"] * case["heads"] * dim * size * case["pools"]
    if op == "copy":
        return {"bytes": case["pairs"] * (2 * page_bytes + 12), "flops": 0}
    if op == "compact":
        moved = case["pages"] * case["used"] * 0.5 * (1 - case["used"] * 0.5)
        return {"bytes": 2 * moved * page_bytes + case["pages"] * 12 + case["seqs"] * case["length"] / case["page"] * 8, "flops": 0}
    # of `children` beams drawn among as many, a share of 1 - 1/e of the last ones goes on; the others are copies
    copied = case["children"] / math.e if case["beams"] else 0
    held = case["length"] / 2 / case["page"]
    return {"bytes": 2 * copied * page_bytes + case["pages"] * 8 + (case["seqs"] + case["children"]) * (held * 4 + 12), "flops": 0}


# ---------------------------------------------------------------- 64-bit values
def exact(case, seed):
    return globals()["_exact_" + case["op"]](prepare(case, seed))


def _exact_attend(s):
    c = s["case"]
    hk, g, dim, page, n = c["kv_heads"], c["group"], c["dim"], c["page"], c["length"]
    out = torch.zeros((c["batch"], hk * g, dim), dtype=torch.float64, device=s["q"].device)
    lse = torch.zeros(out.shape[:2], dtype=torch.float64, device=out.device)
    weights = torch.zeros((c["batch"], hk * g, n), dtype=torch.float64, device=out.device) if c["weights"] else None
    for b, length in enumerate(s["lengths"].tolist()):
        start = max(0, length - c["window"]) if c["window"] else 0
        at = torch.arange(start, length, device=out.device)
        where, slot = s["table"][b].long()[at // page], at % page
        for h in range(hk):
            heads = slice(h * g, (h + 1) * g)
            keys = s["k"][where, h, slot].double()
            scores = s["q"][b, heads].double().mm(keys.t().contiguous()) / math.sqrt(dim)
            lse[b, heads] = torch.logsumexp(scores, 1)
            p = torch.softmax(scores, 1)
            out[b, heads] = p.mm(s["v"][where, h, slot].double())
            if weights is not None:
                weights[b, heads, start:length] = p
    return dict(out=out, lse=lse, weights=weights, status=None)


def _exact_append(s):
    page = s["case"]["page"]
    offsets, lengths, table = s["offsets"].tolist(), s["lengths"].tolist(), s["table"].cpu().numpy()
    pages, slots = [], []
    for b, length in enumerate(lengths):
        for j in range(length - (offsets[b + 1] - offsets[b]), length):
            pages.append(int(table[b, j // page]))
            slots.append(j % page)
    pages, slots = torch.tensor(pages, device=s["k"].device), torch.tensor(slots, device=s["k"].device)
    for h in range(s["case"]["kv_heads"]):
        s["k"][pages, h, slots] = s["k_new"][:, h]
        s["v"][pages, h, slots] = s["v_new"][:, h]
    return dict(k=s["k"], v=s["v"], status=None)


def _moved(pools, moves):
    if moves:
        source, target = (torch.tensor(x, device=pools[0].device) for x in zip(*moves))
        for pool in pools:
            pool.index_copy_(0, target, pool.index_select(0, source))
    return pools


def _exact_fork(s):
    # a sequence at a time, as the words say it: who shares, who copies, which free page comes next
    page = s["case"]["page"]
    table, lengths, refs = s["table"].cpu().numpy(), s["lengths"].tolist(), s["refs"].cpu().numpy().copy()
    parent, new = s["parent"].tolist(), s["n_new"].tolist()
    seen, kinds = set(), []
    for p in parent:
        kinds.append(p >= 0 and p in seen and lengths[p] % page > 0)
        seen.add(p)
    for p, n in enumerate(lengths):
        children = parent.count(p)
        refs[table[p, : n // page]] += children - 1
        if n % page and not children:
            refs[table[p, n // page]] -= 1
    free = np.nonzero(refs <= 0)[0].tolist()
    moves, taken = [], 0
    for p, grow, copies in zip(parent, new, kinds):
        n = lengths[p] if p >= 0 else 0
        need = int(copies) + -(-(n + grow) // page) - -(-n // page)
        if taken + need <= len(free) and copies:
            moves.append((int(table[p, n // page]), free[taken]))
        taken += need
    return dict(table=None, lengths=None, refs=None, status=None, pools=_moved(s["pools"], moves))


def _exact_compact(s):
    live = np.nonzero(s["refs"].cpu().numpy() > 0)[0]
    n = live.size
    holes = np.setdiff1d(np.arange(n), live)
    return dict(table=None, refs=None, map=None, count=None, status=None,
                pools=_moved(s["pools"], list(zip(live[live >= n].tolist(), holes.tolist()))))


def _exact_copy(s):
    return dict(status=None, pools=_moved(s["pools"], list(zip(s["source"].tolist(), s["target"].tolist()))))
