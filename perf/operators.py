"""Measured operators: speculative decoding over the decode step's KV cache.

Each case is one call of one operator: attention of a tree of drafted tokens
over a contiguous or paged cache (every token, or the persisted index set of a
sparse layer), the block tables and slot map of a batch from its lengths, the
append of new K/V rows through a slot map, and the commit of the accepted
drafted rows.  `run` computes the operator from elementary torch operations,
or through the package's entry points where `own` is set.
"""
import math

import torch

own = False
D = 128          # head dim
DEV = "cuda"


# --------------------------------------------------------------------- cases
def listed():
    return [
        # a serving batch of ragged requests, pages of 64 tokens, 16-node trees
        dict(name="tree serving paged", op="tree", batch=32, hq=32, hkv=8, lo=8192, hi=16384,
             tree=16, page=64, k=0, chain=False),
        # one very long context, one KV head per query head, 32-node tree, contiguous cache
        dict(name="tree 100k", op="tree", batch=1, hq=32, hkv=32, lo=102400, hi=102400, tree=32,
             page=0, k=0, chain=False),
        # four long contexts with wide 64-node trees: 256 query rows per KV head
        dict(name="tree wide 32k", op="tree", batch=4, hq=32, hkv=8, lo=30011, hi=32768, tree=64,
             page=0, k=0, chain=False),
        # plain decoding (one token) of a few short chats on pages: latency, the single-token form
        dict(name="tree decode paged", op="tree", batch=4, hq=64, hkv=8, lo=257, hi=2050, tree=1,
             page=16, k=0, chain=True),
        # a sparse layer of the 32K workload with a drafted chain of 5
        dict(name="sparse tree 32k", op="tree", batch=4, hq=32, hkv=8, lo=30011, hi=32768, tree=5,
             page=0, k=2048, chain=True),
        # a sparse layer of the serving batch on pages, 16-node trees
        dict(name="sparse tree serving", op="tree", batch=32, hq=32, hkv=8, lo=8192, hi=16384,
             tree=16, page=64, k=1024, chain=False),
        # a decode step's bookkeeping: every request grows by a draft, some shrink after a rejection
        dict(name="tables decode", op="tables", batch=256, lo=257, hi=16384, new_lo=1, new_hi=9,
             page=16),
        # admission of prompts: tens of thousands of new tokens
        dict(name="tables prompts", op="tables", batch=61, lo=1021, hi=8192, new_lo=1021,
             new_hi=8192, page=32),
        # the drafted rows of a decode step, and the rows of a chunk of prompts
        dict(name="append draft", op="append", tokens=257, hkv=8, page=16, pages=4096),
        dict(name="append prompts", op="append", tokens=32749, hkv=8, page=64, pages=1024),
        # the accepted rows of a batch in every layer
        dict(name="commit small", op="commit", batch=3, hkv=8, layers=4, tree=8, page=16, lo=129,
             hi=2048),
        dict(name="commit serving", op="commit", batch=32, hkv=8, layers=32, tree=32, page=64,
             lo=257, hi=1024),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tree", "tree", "tree", "tables", "append", "commit"])
    page = rng.choice([16, 32, 64, 128])
    if op == "tree":
        hkv = rng.choice([1, 2, 4, 8])
        G = rng.choice([1, 2, 4, 8])
        hi = _log(rng, 64, 32768)
        tree = _log(rng, 1, 64)
        most = min(48, (1 << 21) // (hi * hkv), (1 << 28) // (hi * hkv * G * tree))
        batch = _log(rng, 1, max(1, most))
        k = rng.choice([0, 0, _log(rng, 16, max(17, hi // 4))])
        return dict(op=op, batch=batch, hq=hkv * G, hkv=hkv, lo=max(tree, hi // rng.choice([1, 2, 5])),
                    hi=max(hi, tree), tree=tree, page=rng.choice([0, page]), k=k,
                    chain=rng.random() < 0.4)
    if op == "tables":
        hi = _log(rng, 64, 16384)
        lo = max(1, hi // rng.choice([1, 3, 16]))
        new_hi = _log(rng, 1, lo)
        return dict(op=op, batch=_log(rng, 1, 300 if new_hi < 256 else 40), lo=lo, hi=hi,
                    new_lo=max(1, new_hi // 2), new_hi=new_hi, page=page)
    if op == "append":
        pages = _log(rng, 64, 1024)
        return dict(op=op, tokens=_log(rng, 1, pages * page // 2), hkv=rng.choice([1, 2, 8]),
                    page=page, pages=pages)
    tree = _log(rng, 2, 64)
    return dict(op=op, batch=_log(rng, 1, 32), hkv=rng.choice([1, 2, 8]),
                layers=_log(rng, 1, 16), tree=tree, page=page, lo=max(tree, 65), hi=_log(rng, 128, 1024))


def _lens(case):
    """The lengths of a case before they are shuffled: evenly spread over its range."""
    B, lo, hi = case["batch"], case["lo"], case["hi"]
    return [round(lo + (hi - lo) * (i + 1) / B) for i in range(B)]


def _news(case):
    B, lo, hi = case["batch"], case["new_lo"], case["new_hi"]
    return [min(n, lo + (i * 7919) % (hi - lo + 1)) for i, n in enumerate(_lens(case))]


def work(case):
    op = case["op"]
    if op == "tree":
        B, Hq, Hkv, T, k = (case[x] for x in ("batch", "hq", "hkv", "tree", "k"))
        ctx = [n - T for n in _lens(case)]
        rows = sum((min(c, k) if k else c) + T for c in ctx)
        kv = rows * Hkv * 2 * D * 2
        other = 2 * B * T * Hq * D * 2 + B * T * ((T + 31) // 32) * 4
        if k:
            other += sum(min(c, k) for c in ctx) * Hkv * 4
        if case["page"]:
            other += sum(-(-n // case["page"]) for n in _lens(case)) * 4
        return {"bytes": kv + other, "flops": 4 * D * Hq * T * rows}
    if op == "tables":
        new, pages = sum(_news(case)), sum(-(-n // case["page"]) for n in _news(case))
        return {"bytes": 4 * (case["batch"] * 5 + 3 * pages + new), "flops": 0}
    if op == "append":
        return {"bytes": case["tokens"] * (case["hkv"] * D * 2 * 4 + 4), "flops": 0}
    moved = sum(_accepted_lens(case))
    return {"bytes": moved * (case["hkv"] * case["layers"] * D * 2 * 4 + 4) + 12 * case["batch"],
            "flops": 0}


def _accepted_lens(case):
    T = case["tree"]
    return [1 + (i * 5) % max(1, (T + 1) // 2) for i in range(case["batch"])]


# -------------------------------------------------------------------- inputs
def _tree_mask(parents):
    """[B][T] parents (-1: the context) -> visibility bits int32 [B][T][ceil(T/32)]: a node sees
    its ancestors and itself."""
    B, T = parents.shape
    seen = torch.zeros(B, T, T, dtype=torch.bool)
    at = torch.arange(B)
    for t in range(T):
        p = parents[:, t]
        seen[:, t] = seen[at, p.clamp(min=0)] & (p >= 0)[:, None]
        seen[:, t, t] = True
    W = (T + 31) // 32
    bits = torch.zeros(B, T, W * 32, dtype=torch.int64)
    bits[:, :, :T] = seen
    words = (bits.view(B, T, W, 32) << torch.arange(32)).sum(-1)
    words = torch.where(words >= 1 << 31, words - (1 << 32), words)
    return words.to(torch.int32)


def _prepare_tree(case, gen, cpu):
    B, Hq, Hkv, T, page, k = (case[x] for x in ("batch", "hq", "hkv", "tree", "page", "k"))
    lens = torch.tensor(_lens(case))[torch.randperm(B, generator=cpu)]
    N = max(case["hi"], T)
    s = dict(case=case, T=T, N=N)
    if page:
        blocks = -(-N // page)
        P = B * blocks
        s["table"] = torch.randperm(P, generator=cpu).view(B, blocks).to(torch.int32).to(DEV)
        dims = (P, Hkv, page, D)
    else:
        s["table"] = None
        dims = (B, Hkv, N, D)
    s["k"] = torch.randn(dims, generator=gen, device=DEV, dtype=torch.bfloat16)
    s["v"] = torch.randn(dims, generator=gen, device=DEV, dtype=torch.bfloat16)
    # queries a little longer than unit length: a peaked softmax, as trained heads have
    s["q"] = (2 * torch.randn(B, T, Hq, D, generator=gen, device=DEV)).to(torch.bfloat16)
    # a drafted token continues one of the last few nodes, or the context
    back = torch.randint(1, 5, (B, T), generator=cpu)
    s["mask"] = None
    if not case["chain"]:
        s["mask"] = _tree_mask((torch.arange(T)[None] - back).clamp(min=-1)).to(DEV)
    # most requests draft a full tree, some a smaller one
    small = torch.randint(1, T + 1, (B,), generator=cpu)
    tl = torch.where(torch.rand(B, generator=cpu) < 0.8, torch.full((B,), T), small)
    s["tree_lens"] = tl.to(torch.int32).to(DEV)
    s["seq_lens"] = lens.to(torch.int32).to(DEV)
    s["idx"] = None
    if k:
        # distinct random positions of the context, ascending, -1 padded
        ctx = (lens - tl).to(DEV)
        r = torch.rand(B, Hkv, N, generator=gen, device=DEV)
        r = torch.where(torch.arange(N, device=DEV) < ctx[:, None, None], r, 2.0)
        val, pos = r.topk(min(k, N), dim=-1, largest=False)
        pos = torch.where(val < 2.0, pos, N).sort(-1).values
        pos = torch.where(pos < N, pos, -1).to(torch.int32)
        s["idx"] = pos.contiguous()
    s["out"] = torch.zeros(B, T, Hq, D, dtype=torch.bfloat16, device=DEV)
    if own:
        import sparse_attention_td_gb300 as td
        s["shape"] = td.make_shape(B, Hq, Hkv, N)
        s["cache"] = td.make_cache(s["k"], s["v"], s["table"])
        s["ws"] = td.Workspace(s["shape"], 0, tree_size=T)
    return s


def _prepare_tables(case, gen, cpu):
    B, page = case["batch"], case["page"]
    order = torch.randperm(B, generator=cpu)
    lens, new = torch.tensor(_lens(case))[order], torch.tensor(_news(case))[order]
    blocks = -(-case["hi"] // page) + 1
    target = (lens + page - 1) // page
    held = (lens - new + page - 1) // page
    # a request in eight holds pages that a rejected draft left over
    over = (torch.rand(B, generator=cpu) < 0.125) & (new < 16)
    held = torch.where(over, (target + 1).clamp(max=blocks), held)
    P = int(target.sum()) + B + 64
    ids = torch.randperm(P, generator=cpu)
    table = torch.full((B, blocks), -1, dtype=torch.int64)
    own_it = torch.arange(blocks)[None] < held[:, None]
    n = int(held.sum())
    table[own_it] = ids[:n]
    free = torch.full((P,), -1, dtype=torch.int64)
    free[: P - n] = ids[n:]
    i32 = lambda x: x.to(torch.int32).to(DEV)
    total = int(new.sum())
    s = dict(case=case, table=i32(table), held=i32(held), free=i32(free),
             count=i32(torch.tensor([P - n])), seq_lens=i32(lens), new_lens=i32(new), page=page,
             max_new=total + 13)    # a padded step: the last slots belong to no token
    s["held_out"], s["count_out"] = torch.zeros_like(s["held"]), torch.zeros_like(s["count"])
    s["cu"] = torch.zeros(B + 1, dtype=torch.int32, device=DEV)
    s["slots"] = torch.zeros(s["max_new"], dtype=torch.int32, device=DEV)
    if own:
        import sparse_attention_td_gb300 as td
        s["ws"] = td.Workspace(td.make_shape(1, 1, 1, 1), 0)
    return s


def _prepare_append(case, gen, cpu):
    n, Hkv, page, P = (case[x] for x in ("tokens", "hkv", "page", "pages"))
    s = dict(case=case)
    # one page more than the cache has: where the plain form sends padding slots
    s["k_all"], s["v_all"] = (torch.randn(P + 1, Hkv, page, D, generator=gen, device=DEV,
                                          dtype=torch.bfloat16) for _ in range(2))
    s["k"], s["v"] = s["k_all"][:P], s["v_all"][:P]
    # the K and V columns of a packed projection: rows of 2 * Hkv * D values
    s["kv_new"] = torch.randn(n, 2, Hkv, D, generator=gen, device=DEV, dtype=torch.bfloat16)
    # runs of positions inside random pages, a few padding slots
    order = torch.randperm(P, generator=cpu)
    slots = (order[:, None] * page + torch.arange(page)).view(-1)[:n].clone()
    slots[torch.rand(n, generator=cpu) < 0.01] = -1
    s["slots"] = slots.to(torch.int32).to(DEV)
    if own:
        import sparse_attention_td_gb300 as td
        s["shape"] = td.make_shape(1, Hkv, Hkv, P * page)
        s["cache"] = td.make_cache(s["k"], s["v"])
    return s


def _prepare_commit(case, gen, cpu):
    B, Hkv, L, T, page = (case[x] for x in ("batch", "hkv", "layers", "tree", "page"))
    N = max(case["hi"], T)
    blocks = -(-N // page)
    P = B * blocks
    s = dict(case=case)
    s["k"] = torch.randn(L, P, Hkv, page, D, generator=gen, device=DEV, dtype=torch.bfloat16)
    s["v"] = torch.randn(L, P, Hkv, page, D, generator=gen, device=DEV, dtype=torch.bfloat16)
    s["table"] = torch.randperm(P, generator=cpu).view(B, blocks).to(torch.int32).to(DEV)
    order = torch.randperm(B, generator=cpu)
    s["seq_lens"] = torch.tensor(_lens(case)).clamp(min=T)[order].to(torch.int32).to(DEV)
    s["tree_lens"] = torch.full((B,), T, dtype=torch.int32, device=DEV)
    acc = torch.tensor(_accepted_lens(case))[order]
    # a root-to-leaf path: ascending node numbers
    r = torch.rand(B, T, generator=cpu).argsort(1)
    r = torch.where(torch.arange(T)[None] < acc[:, None], r, T).sort(1).values
    s["accepted"] = torch.where(r < T, r, -1).to(torch.int32).to(DEV)
    s["accepted_lens"] = acc.to(torch.int32).to(DEV)
    s["seq_out"] = torch.zeros(B, dtype=torch.int32, device=DEV)
    if own:
        import sparse_attention_td_gb300 as td
        s["shape"] = td.make_shape(B, Hkv, Hkv, N)
        s["caches"] = [td.make_cache(s["k"][l], s["v"][l], s["table"]) for l in range(L)]
        s["ws"] = td.Workspace(s["shape"], 0)
    return s


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    cpu = torch.Generator().manual_seed(seed)
    return {"tree": _prepare_tree, "tables": _prepare_tables, "append": _prepare_append,
            "commit": _prepare_commit}[case["op"]](case, gen, cpu)


# --------------------------------------------------------------- plain forms
def _positions(x, table, pos):
    """Rows [B][Hkv][n][D] of positions pos [B][Hkv][n] (clamped by the caller)."""
    B, Hkv = pos.shape[:2]
    h = torch.arange(Hkv, device=DEV)[None, :, None]
    b = torch.arange(B, device=DEV)[:, None, None]
    if table is None:
        return x[b, h, pos]
    page = x.shape[2]
    return x[table.long()[b, pos // page], h, pos % page]


def _plain_tree(s):
    q, k, v, T, N = s["q"], s["k"], s["v"], s["T"], s["N"]
    B, _, Hq, _ = q.shape
    Hkv = k.shape[1]
    G = Hq // Hkv
    n_t = s["tree_lens"].long()
    ctx = s["seq_lens"].long() - n_t
    nodes = torch.arange(T, device=DEV)
    at = (ctx[:, None] + nodes).clamp(max=N - 1)[:, None].expand(B, Hkv, T)
    if s["idx"] is None:
        if s["table"] is None:
            kc, vc = k, v
        else:
            kc, vc = (x[s["table"].long()].transpose(1, 2).reshape(B, Hkv, -1, D) for x in (k, v))
        seen = (torch.arange(kc.shape[2], device=DEV) < ctx[:, None])[:, None]      # [B][1][n]
    else:
        idx = s["idx"].long()
        kc, vc = (_positions(x, s["table"], idx.clamp(min=0)) for x in (k, v))
        seen = (idx >= 0) & (idx < ctx[:, None, None])
    kt, vt = (_positions(x, s["table"], at) for x in (k, v))
    qf = q.float().view(B, T, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, T * G, D)
    scale = 1 / math.sqrt(D)
    a = (qf @ kc.float().transpose(2, 3)) * scale
    a = a.masked_fill(~seen[:, :, None], float("-inf"))
    t = (qf @ kt.float().transpose(2, 3)) * scale
    if s["mask"] is None:
        bits = (nodes[None, :] <= nodes[:, None])[None]
    else:
        bits = ((s["mask"][:, :, nodes // 32].long() >> (nodes % 32)) & 1).bool()
    bits = bits & (nodes[None, None] < n_t[:, None, None])
    t = t.masked_fill(~bits.repeat_interleave(G, 1)[:, None], float("-inf"))
    m = torch.maximum(a.amax(-1), t.amax(-1))[..., None]
    m = torch.where(m == float("-inf"), 0.0, m)
    a, t = (a - m).exp_(), (t - m).exp_()
    l = a.sum(-1) + t.sum(-1)
    o = (a @ vc.float() + t @ vt.float()) / torch.where(l > 0, l, 1.0)[..., None]
    o = o.view(B, Hkv, T, G, D).permute(0, 2, 1, 3, 4).reshape(B, T, Hq, D)
    return torch.where((nodes < n_t[:, None])[..., None, None], o.to(torch.bfloat16), s["out"])


def _plain_tables(s):
    page, table, free = s["page"], s["table"].long(), s["free"].long()
    B, blocks = table.shape
    P = free.numel()
    lens, new, held = s["seq_lens"].long(), s["new_lens"].long(), s["held"].long()
    target = (lens + page - 1) // page
    j = torch.arange(blocks, device=DEV)
    back = (j >= target[:, None]) & (j < held[:, None])
    rank = back.view(-1).cumsum(0) - 1
    at = torch.where(back.view(-1), s["count"].long() + rank, P)
    stack = torch.cat([free, free.new_zeros(1)]).scatter(0, at, table.view(-1))[:P]
    top = s["count"].long() + back.sum()
    need = (target - held).clamp(min=0)
    fits = need.cumsum(0) <= top
    take = (j >= held[:, None]) & (j < target[:, None])
    rank = (take.view(-1).cumsum(0) - 1).view(B, blocks)
    take = take & fits[:, None]
    table = torch.where(take, stack[(top - 1 - rank).clamp(min=0, max=P - 1)], table)
    held = torch.where(fits | (need == 0), target, held)
    count = top - (need * fits).sum()
    cu = torch.cat([new.new_zeros(1), new.cumsum(0)])
    i = torch.arange(s["max_new"], device=DEV)
    b = (torch.searchsorted(cu, i, right=True) - 1).clamp(max=B - 1)
    p = (lens[b] - new[b] + i - cu[b]).clamp(max=blocks * page - 1)
    slot = table[b, p // page] * page + p % page
    slot = torch.where((i < cu[-1]) & (p // page < held[b]), slot, -1)
    return [x.to(torch.int32) for x in (table, held, stack, count, cu, slot)]


def _plain_append(s):
    kv, page = s["kv_new"], s["k"].shape[2]
    slot = s["slots"].long()
    at = torch.where(slot >= 0, slot, s["k"].shape[0] * page)
    s["k_all"][at // page, :, at % page] = kv[:, 0]
    s["v_all"][at // page, :, at % page] = kv[:, 1]
    return [s["k"], s["v"]]


def _plain_commit(s):
    k, v, table = s["k"], s["v"], s["table"].long()
    page = k.shape[3]
    B, T = s["accepted"].shape
    ctx = s["seq_lens"].long() - s["tree_lens"].long()
    i = torch.arange(T, device=DEV)
    keep = i < s["accepted_lens"].long()[:, None]
    src = torch.where(keep, s["accepted"].long(), i) + ctx[:, None]     # others stay where they are
    dst = (i + ctx[:, None])
    b = torch.arange(B, device=DEV)[:, None]
    sp, dp = table[b, src // page], table[b, dst // page]
    for x in (k, v):
        x[:, dp, :, dst % page] = x[:, sp, :, src % page]
    return [k, v, (ctx + s["accepted_lens"].long()).to(torch.int32)]


def run(s):
    op = s["case"]["op"]
    if not own:
        return {"tree": _plain_tree, "tables": _plain_tables, "append": _plain_append,
                "commit": _plain_commit}[op](s)
    import sparse_attention_td_gb300 as td
    if op == "tree":
        if s["idx"] is None:
            td.td_tree_attn(s["shape"], s["cache"], s["T"], s["tree_lens"], s["mask"], s["q"],
                            s["seq_lens"], s["out"], ws=s["ws"])
        else:
            td.td_tree_sparse_attn(s["shape"], s["cache"], s["T"], s["tree_lens"], s["mask"],
                                   s["q"], s["seq_lens"], s["idx"], s["case"]["k"], s["out"],
                                   ws=s["ws"])
        return s["out"]
    if op == "tables":
        td.td_block_tables(s["seq_lens"], s["new_lens"], s["page"], s["table"], s["held"],
                           s["held_out"], s["free"], s["count"], s["count_out"], s["cu"],
                           s["slots"], ws=s["ws"])
        return [s["table"], s["held_out"], s["free"], s["count_out"], s["cu"], s["slots"]]
    if op == "append":
        td.td_kv_append_slots(s["shape"], s["cache"], s["kv_new"][:, 0], s["kv_new"][:, 1],
                              s["slots"])
        return [s["k"], s["v"]]
    td.td_tree_commit(s["shape"], s["caches"], s["case"]["tree"], s["tree_lens"], s["accepted"],
                      s["accepted_lens"], s["seq_lens"], s["seq_out"], ws=s["ws"])
    return [s["k"], s["v"], s["seq_out"]]


# ---------------------------------------------------------------- 64 bits
def exact(case, seed):
    """Attention from its definition in 64 bits, one (request, KV head) at a time.  The other
    operators move whole values: nothing is computed."""
    if case["op"] != "tree":
        return None
    s = prepare(case, seed)
    B, Hq, Hkv, T = case["batch"], case["hq"], case["hkv"], case["tree"]
    G, page = Hq // Hkv, case["page"]
    out = torch.zeros(B, T, Hq, D, dtype=torch.float64, device=DEV)
    lens, sizes = s["seq_lens"].tolist(), s["tree_lens"].tolist()
    for b in range(B):
        n, nt = lens[b], sizes[b]
        c = n - nt
        sees = torch.ones(nt, nt, dtype=torch.bool, device=DEV).tril()
        if s["mask"] is not None:
            words = s["mask"][b, :nt].long() & 0xFFFFFFFF
            sees = torch.stack([(words[:, j // 32] >> (j % 32)) & 1 for j in range(nt)], 1).bool()
        for g in range(Hkv):
            if page:
                ids = s["table"][b, : -(-n // page)].long()
                kr, vr = s["k"][ids, g].reshape(-1, D)[:n], s["v"][ids, g].reshape(-1, D)[:n]
            else:
                kr, vr = s["k"][b, g, :n], s["v"][b, g, :n]
            rows = torch.arange(c, device=DEV)
            if s["idx"] is not None:
                rows = s["idx"][b, g].long()
                rows = rows[(rows >= 0) & (rows < c)]
            allowed = torch.cat([torch.ones(nt, rows.numel(), dtype=torch.bool, device=DEV), sees], 1)
            rows = torch.cat([rows, torch.arange(c, n, device=DEV)])
            kd, vd = kr[rows].double(), vr[rows].double()
            qd = s["q"][b, :nt, g * G:(g + 1) * G].double()
            z = torch.einsum("tgd,nd->tgn", qd, kd) / D ** 0.5
            z = z.masked_fill(~allowed[:, None], -math.inf)
            out[b, :nt, g * G:(g + 1) * G] = torch.einsum("tgn,nd->tgd", torch.softmax(z, -1), vd)
    return out
