"""Measured operators of small caches: windows with sinks, 4-bit rows, eviction.

Each case is one call of one operator: attention with a sliding window and a
few first tokens that stay visible (prompts, chunks and single tokens), the
append of rows into a 4-bit cache and the attention over it (prompts, single
tokens, a persisted index set), attention that adds its probabilities to a
weight per cached position, and the eviction of the lightest positions.
`run` computes the operator from elementary torch operations, or through the
package's entry points where `own` is set.
"""
import math

import torch

own = False
D = 128          # head dim
DEV = "cuda"
CHUNK = 128      # query tokens of one block of the plain form


# --------------------------------------------------------------------- cases
def listed():
    return [
        # a batch of prompts through a windowed layer, ragged, pages of 64 tokens: the largest product
        dict(name="window prompts", op="attn", batch=5, hq=32, hkv=8, lo=1021, hi=6144, new_lo=1021,
             new_hi=6144, window=1024, sinks=4, page=64, q4=False, k=0),
        # a serving batch decoding: one token per request, a window much shorter than the requests
        dict(name="window decode", op="attn", batch=32, hq=32, hkv=8, lo=8192, hi=16384, new_lo=0,
             new_hi=0, window=4096, sinks=4, page=64, q4=False, k=0),
        # single tokens and small chunks of prompts in one step, grouped queries of 8, small pages
        dict(name="window mixed", op="attn", batch=9, hq=64, hkv=8, lo=257, hi=8191, new_lo=1,
             new_hi=61, window=1023, sinks=16, page=16, q4=False, k=0),
        # the serving batch over a 4-bit cache
        dict(name="q4 decode", op="attn", batch=32, hq=32, hkv=8, lo=8192, hi=16384, new_lo=0, new_hi=0,
             window=0, sinks=0, page=64, q4=True, k=0),
        # chunks of prompts on long contexts held in 4 bits
        dict(name="q4 prompts", op="attn", batch=3, hq=32, hkv=8, lo=5003, hi=16384, new_lo=517,
             new_hi=1024, window=0, sinks=0, page=32, q4=True, k=0),
        # a sparse layer of the 32K workload over a contiguous 4-bit cache
        dict(name="q4 sparse 32k", op="attn", batch=4, hq=32, hkv=8, lo=30011, hi=32768, new_lo=0,
             new_hi=0, window=0, sinks=0, page=0, q4=True, k=2048),
        # the rows of a step's prompts, and of its single tokens, into a 4-bit cache
        dict(name="q4 append prompts", op="append", tokens=32749, hkv=8, page=64, pages=1024),
        dict(name="q4 append tokens", op="append", tokens=257, hkv=8, page=16, pages=512),
        # a decoding batch whose caches are kept at about 4K positions, and a few short chats
        dict(name="weights serving", op="weights", batch=32, hq=32, hkv=8, lo=1025, hi=4224, page=64,
             fresh=1),
        dict(name="weights chats", op="weights", batch=3, hq=16, hkv=8, lo=257, hi=2050, page=0, fresh=1),
        # the caches of a decoding batch back to 4096 positions, in place
        dict(name="evict decode", op="evict", batch=32, hkv=8, lo=4097, hi=4224, budget=4096, sinks=4,
             recent=1024, page=64, place=True),
        # long prompts into small caches of their own
        dict(name="evict prompts", op="evict", batch=7, hkv=8, lo=9001, hi=16384, budget=2048, sinks=4,
             recent=509, page=32, place=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "attn", "append", "weights", "evict"])
    page = rng.choice([0, 8, 16, 32, 64, 128, 48])
    hkv, G = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 8])
    if op == "append":
        pages, page = _log(rng, 64, 1024), page or 16
        return dict(op=op, tokens=_log(rng, 1, min(32749, pages * page // 2)), hkv=hkv, page=page, pages=pages)
    if op == "evict":
        hi = _log(rng, 64, 16384)
        budget = _log(rng, 32, hi)
        sinks = rng.choice([0, 1, 4, 16])
        most = max(1, min(32, (1 << 18) // (hi * hkv) * 4))
        return dict(op=op, batch=_log(rng, 1, most), hkv=hkv, lo=max(1, hi // rng.choice([1, 2, 3])), hi=hi,
                    budget=budget, sinks=min(sinks, budget // 2), recent=_log(rng, 1, max(2, budget // 2)),
                    page=page, place=rng.random() < 0.5)
    q4 = rng.random() < 0.5 and op == "attn"
    kind = rng.choice(["one", "one", "prompts", "sparse"]) if op == "attn" else "one"
    hi = _log(rng, 64, 8192 if op == "weights" else 16384)
    lo = max(1, hi // rng.choice([1, 2, 5]))
    if kind == "sparse":
        q4 = True
    if kind == "prompts":
        new_hi = _log(rng, 1, min(hi, 2048))
        batch = _log(rng, 1, 8)
    else:
        new_hi = 0
        batch = _log(rng, 1, max(1, min(48, (1 << 21) // (hi * hkv))))
    window = rng.choice([0, _log(rng, 1, hi), _log(rng, 16, max(17, hi // 2))]) if kind != "sparse" else 0
    keys = min(hi, window + new_hi + 64) if window else hi
    while kind == "prompts" and batch > 1 and batch * (new_hi + CHUNK) * hkv * G * keys > 1 << 29:
        batch //= 2
    while kind == "prompts" and batch * (new_hi + CHUNK) * hkv * G * keys > 1 << 29:
        new_hi = max(1, new_hi // 2)
    if op == "weights":
        return dict(op=op, batch=batch, hq=hkv * G, hkv=hkv, lo=lo, hi=hi, page=page,
                    fresh=rng.choice([1, 1, _log(rng, 1, hi)]))
    return dict(op=op, batch=batch, hq=hkv * G, hkv=hkv, lo=lo, hi=hi, new_lo=min(new_hi, 1), new_hi=new_hi,
                window=window, sinks=rng.choice([0, 1, 4, 33]) if window else 0, page=page, q4=q4,
                k=_log(rng, 16, max(17, hi // 4)) if kind == "sparse" else 0)


def _lens(case):
    """The lengths of a case before they are shuffled: evenly spread over its range."""
    B, lo, hi = case["batch"], case["lo"], case["hi"]
    return [round(lo + (hi - lo) * (i + 1) / B) for i in range(B)]


def _news(case):
    """New tokens of each request; none given: one each."""
    lo, hi = case["new_lo"], case["new_hi"]
    return [min(n, lo + (i * 7919 + hi - lo) % (hi - lo + 1)) if hi else 1 for i, n in enumerate(_lens(case))]


def _row_bytes(q4):
    """One token's K and V of one KV head."""
    return 2 * (D // 2 + D // 16) if q4 else 2 * D * 2


def work(case):
    op, hkv = case["op"], case["hkv"]
    if op == "append":
        return {"bytes": case["tokens"] * (hkv * (2 * D * 2 + _row_bytes(True)) + 4), "flops": 0}
    lens, page = _lens(case), case["page"]
    tables = 4 * sum(-(-n // page) for n in lens) if page else 0
    if op == "evict":
        # what a first pass moves: the kept rows behind the first ones; and the weights
        kept = [min(n, case["budget"]) for n in lens]
        rows = [k if not case["place"] else (k - case["sinks"] if n > k else 0) for k, n in zip(kept, lens)]
        return {"bytes": hkv * (sum(rows) * 2 * _row_bytes(False) + 4 * sum(lens) + 8 * sum(kept)) + tables, "flops": 0}
    hq = case["hq"]
    if op == "weights":
        return {"bytes": sum(lens) * hkv * (_row_bytes(False) + 8) + 4 * D * hq * case["batch"] + tables,
                "flops": 4 * D * hq * sum(lens)}
    news, W, S, k = _news(case), case["window"], case["sinks"], case["k"]
    pairs = rows = 0
    for n, t in zip(lens, news):
        if k:
            pairs, rows = pairs + min(n, k), rows + min(n, k)
        elif not W:
            pairs, rows = pairs + t * n - t * (t - 1) // 2, rows + n
        else:
            # a query at position p sees min(p + 1, W) recent ones and the first ones before those
            pairs += sum(min(p + 1, W) + min(S, max(0, p + 1 - W)) for p in range(n - t, n))
            low = max(0, n - t - W + 1)
            rows += n - low + min(S, low)
    return {"bytes": rows * hkv * _row_bytes(case["q4"]) + 4 * D * hq * sum(news) + tables +
            (4 * hkv * rows if k else 0), "flops": 4 * D * hq * pairs}


# -------------------------------------------------------------------- inputs
def _quantise(x):
    """bf16 rows [..., 128] -> codes uint8 [..., 64] (even value in the low half) and scales uint8
    [..., 8]: e2m1 codes of x / s, s the e4m3 value nearest to a 16th's largest magnitude / 6.
    Quotients of these short numbers are on the right side of every border in fp32."""
    y = x.float().view(*x.shape[:-1], 8, 16)
    s = (y.abs().amax(-1, keepdim=True) / 6).clamp(max=448).to(torch.float8_e4m3fn)
    sf = s.float()
    t = y.abs() / torch.where(sf > 0, sf, 1.0)
    code = ((t > 0.25).to(torch.uint8) + (t >= 0.75) + (t > 1.25) + (t >= 1.75) + (t > 2.5) +
            (t >= 3.5) + (t > 5)) * (sf > 0)
    code = (code.to(torch.uint8) | (torch.signbit(y).to(torch.uint8) << 3)).view(*x.shape[:-1], 64, 2)
    return code[..., 0] | (code[..., 1] << 4), s.squeeze(-1).view(torch.uint8)


def _values(codes, scales, dtype):
    """The values that 4-bit rows stand for."""
    grid = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], dtype=dtype, device=DEV)
    pair = torch.stack([codes & 15, codes >> 4], -1).int()
    s = scales.contiguous().view(torch.float8_e4m3fn).to(dtype)
    return (grid[pair].view(*codes.shape[:-1], 8, 16) * s[..., None]).flatten(-2)


def _rows(gen, *dims):
    return torch.randn(*dims, D, generator=gen, device=DEV, dtype=torch.bfloat16)


def _geometry(case, cpu):
    """(pages, page size, block table) of a cache for the case's requests."""
    B, hi, page = case["batch"], case["hi"], case["page"]
    if not page:
        return B, hi, None
    blocks = -(-hi // page)
    return B * blocks, page, torch.randperm(B * blocks, generator=cpu).view(B, blocks).to(torch.int32).to(DEV)


def _prepare_attn(case, gen, cpu):
    B, Hq, Hkv, N = (case[x] for x in ("batch", "hq", "hkv", "hi"))
    order = torch.randperm(B, generator=cpu)
    lens, new = torch.tensor(_lens(case))[order], torch.tensor(_news(case))[order]
    P, page, table = _geometry(case, cpu)
    s = dict(case=case, table=table, seq_lens=lens.to(torch.int32).to(DEV), N=N)
    total = int(new.sum())
    # queries a little longer than unit length: a peaked softmax, as trained heads have
    s["q"] = (2 * torch.randn(total, Hq, D, generator=gen, device=DEV)).to(torch.bfloat16)
    s["cu"] = torch.cat([new.new_zeros(1), new.cumsum(0)]).to(torch.int32).to(DEV)
    # the blocks of query tokens that a step's scheduler would cut: (request, first token, tokens)
    s["blocks"] = torch.tensor([(b, t, min(CHUNK, n - t)) for b, n in enumerate(new.tolist())
                                for t in range(0, n, CHUNK)], device=DEV)
    k, v = _rows(gen, P, Hkv, page), _rows(gen, P, Hkv, page)
    if case["q4"]:
        (s["k"], ks), (s["v"], vs) = _quantise(k), _quantise(v)
        s["scales"] = torch.cat([ks, vs], -1)
    else:
        s["k"], s["v"] = k, v
    s["idx"] = None
    if case["k"]:
        # distinct random positions, ascending, -1 padded
        r = torch.rand(B, Hkv, N, generator=gen, device=DEV)
        r = torch.where(torch.arange(N, device=DEV) < s["seq_lens"][:, None, None], r, 2.0)
        val, pos = r.topk(min(case["k"], N), dim=-1, largest=False)
        pos = torch.where(val < 2.0, pos, N).sort(-1).values
        s["idx"] = torch.where(pos < N, pos, -1).to(torch.int32).contiguous()
    s["out"] = torch.zeros_like(s["q"])
    if own:
        import sparse_attention_td_gb300 as td
        s["shape"] = td.make_shape(B, Hq, Hkv, N)
        s["cache"] = (td.make_q4_cache(s["k"], s["v"], s["scales"], table) if case["q4"] else
                      td.make_cache(s["k"], s["v"], table))
        s["ws"] = td.Workspace(s["shape"], 0, cache_calls=True)
    return s


def _prepare_append(case, gen, cpu):
    n, Hkv, page, P = (case[x] for x in ("tokens", "hkv", "page", "pages"))
    # the K and V columns of a packed projection; a few channels are much larger, as trained keys have
    kv = torch.randn(n, 2, Hkv, D, generator=gen, device=DEV)
    kv *= torch.exp(1.5 * torch.randn(Hkv, D, generator=gen, device=DEV))
    s = dict(case=case, kv_new=kv.to(torch.bfloat16))
    # one page more than the cache has: where the plain form sends padding slots
    byte = lambda w: torch.randint(0, 120, (P + 1, Hkv, page, w), generator=gen, device=DEV, dtype=torch.uint8)
    s["k_all"], s["v_all"], s["s_all"] = byte(D // 2), byte(D // 2), byte(D // 8)
    s["k"], s["v"], s["scales"] = (s[x][:P] for x in ("k_all", "v_all", "s_all"))
    # runs of positions inside random pages, a few padding slots
    order = torch.randperm(P, generator=cpu)
    slots = (order[:, None] * page + torch.arange(page)).view(-1)[:n].clone()
    slots[torch.rand(n, generator=cpu) < 0.01] = -1
    s["slots"] = slots.to(torch.int32).to(DEV)
    if own:
        import sparse_attention_td_gb300 as td
        s["shape"] = td.make_shape(1, Hkv, Hkv, P * page)
        s["cache"] = td.make_q4_cache(s["k"], s["v"], s["scales"])
    return s


def _prepare_weights(case, gen, cpu):
    B, Hq, Hkv, N = (case[x] for x in ("batch", "hq", "hkv", "hi"))
    P, page, table = _geometry(case, cpu)
    lens = torch.tensor(_lens(case))[torch.randperm(B, generator=cpu)]
    s = dict(case=case, table=table, N=N, seq_lens=lens.to(torch.int32).to(DEV))
    s["k"], s["v"] = _rows(gen, P, Hkv, page), _rows(gen, P, Hkv, page)
    s["q"] = (2 * torch.randn(B, Hq, D, generator=gen, device=DEV)).to(torch.bfloat16)
    # what earlier steps have added up: a few heavy positions
    s["weights"] = torch.exp(2 * torch.randn(B, Hkv, N, generator=gen, device=DEV) - 4)
    s["logits"] = torch.zeros(B, Hq, N, device=DEV)
    s["out"] = torch.zeros_like(s["q"])
    if own:
        import sparse_attention_td_gb300 as td
        s["shape"] = td.make_shape(B, Hq, Hkv, N)
        s["cache"] = td.make_cache(s["k"], s["v"], table)
        s["ws"] = td.Workspace(s["shape"], 0, cache_calls=True)
    return s


def _prepare_evict(case, gen, cpu):
    B, Hkv, N, budget = (case[x] for x in ("batch", "hkv", "hi", "budget"))
    P, page, table = _geometry(case, cpu)
    lens = torch.tensor(_lens(case))[torch.randperm(B, generator=cpu)]
    s = dict(case=case, table=table, N=N, seq_lens=lens.to(torch.int32).to(DEV))
    s["k"], s["v"] = _rows(gen, P, Hkv, page), _rows(gen, P, Hkv, page)
    s["weights"] = torch.exp(2 * torch.randn(B, Hkv, N, generator=gen, device=DEV) - 4)
    if case["place"]:
        s["to_k"], s["to_v"], s["to_table"], s["to_weights"] = s["k"], s["v"], table, s["weights"]
    else:
        P2, page2, s["to_table"] = _geometry(dict(case, hi=budget), cpu)
        s["to_k"], s["to_v"] = (torch.zeros(P2, Hkv, page2, D, device=DEV, dtype=torch.bfloat16) for _ in range(2))
        s["to_weights"] = torch.zeros(B, Hkv, budget, device=DEV)
    s["kept"] = torch.full((B, Hkv, budget), -1, dtype=torch.int32, device=DEV)
    s["seq_out"] = torch.zeros(B, dtype=torch.int32, device=DEV)
    if own:
        import sparse_attention_td_gb300 as td
        s["shape"] = td.make_shape(B, Hkv, Hkv, N)
        s["cache"] = td.make_cache(s["k"], s["v"], table)
        s["to"] = s["cache"] if case["place"] else td.make_cache(s["to_k"], s["to_v"], s["to_table"])
        s["ws"] = td.Workspace(s["shape"], 0)
    return s


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    cpu = torch.Generator().manual_seed(seed)
    return {"attn": _prepare_attn, "append": _prepare_append, "weights": _prepare_weights,
            "evict": _prepare_evict}[case["op"]](case, gen, cpu)


# --------------------------------------------------------------- plain forms
def _at(x, table, b, pos):
    """Rows [n][Hkv][m][...] of positions pos [n][Hkv or 1][m] of requests b [n]."""
    h = torch.arange(x.shape[1], device=DEV)[None, :, None]
    if table is None:
        return x[b[:, None, None], h, pos]
    page = x.shape[2]
    return x[table.long()[b[:, None, None], pos // page], h, pos % page]


def _cached(s, b, pos, dtype):
    """K and V of positions, as numbers."""
    k, v = _at(s["k"], s["table"], b, pos), _at(s["v"], s["table"], b, pos)
    if not s["case"].get("q4"):
        return k.to(dtype), v.to(dtype)
    sc = _at(s["scales"], s["table"], b, pos)
    return _values(k, sc[..., :8], dtype), _values(v, sc[..., 8:], dtype)


def _softmax_parts(z):
    m = z.amax(-1, keepdim=True)
    e = torch.exp(z - torch.where(m == -math.inf, 0.0, m))
    return e, e.sum(-1, keepdim=True)


def _plain_attn(s):
    c, q = s["case"], s["q"]
    Hq, Hkv, W, S = c["hq"], c["hkv"], c["window"], c["sinks"]
    G, N = Hq // Hkv, s["N"]
    b, first, count = s["blocks"].unbind(1)
    M = CHUNK if c["new_hi"] else 1
    lens, cu = s["seq_lens"].long(), s["cu"].long()
    t = torch.arange(M, device=DEV)
    row = (cu[b] + first)[:, None] + t                                        # [n][M] rows of q
    there = t < count[:, None]
    p = (lens[b] - (cu[b + 1] - cu[b]) + first)[:, None] + t                  # positions
    if s["idx"] is not None:
        pos = s["idx"].long()[b]
        seen = (pos >= 0)[:, :, None]                                         # [n][Hkv][1][m]
        pos = pos.clamp(min=0)
    else:
        m = min(N, S + W + M - 1) if W else N
        if m < N:
            # the first tokens, then the windows of the block's tokens
            low = (p[:, 0] - W + 1).clamp(min=S)
            j = torch.arange(m, device=DEV)[None]
            pos = torch.where(j < S, j, low[:, None] + j - S)[:, None]
        else:
            pos = torch.arange(m, device=DEV)[None, None].expand(b.numel(), 1, m)
        seen = pos[:, :, None] <= p[:, None, :, None]                         # [n][1][M][m]
        if W:
            seen = seen & ((pos[:, :, None] < S) | (p[:, None, :, None] - pos[:, :, None] < W))
        pos = pos.clamp(max=N - 1)
    k, v = _cached(s, b, pos, torch.float32)                                  # [n][Hkv][m][D]
    qb = q[row.clamp(max=q.shape[0] - 1)].float().view(-1, M, Hkv, G, D).permute(0, 2, 3, 1, 4)
    z = (qb.reshape(-1, Hkv, G * M, D) @ k.transpose(2, 3)) * (1 / math.sqrt(D))
    z = z.view(-1, Hkv, G, M, k.shape[2]).masked_fill_(~seen[:, :, None], -math.inf)
    e, l = _softmax_parts(z)
    o = (e.view(-1, Hkv, G * M, k.shape[2]) @ v).view(-1, Hkv, G, M, D) / torch.where(l > 0, l, 1.0)
    o = o.permute(0, 3, 1, 2, 4).reshape(-1, M, Hq, D).to(torch.bfloat16)
    s["out"][row[there]] = o[there]
    return s["out"]


def _plain_append(s):
    page = s["k"].shape[2]
    slot = s["slots"].long()
    at = torch.where(slot >= 0, slot, s["k"].shape[0] * page)
    codes, scales = _quantise(s["kv_new"])
    s["k_all"][at // page, :, at % page] = codes[:, 0]
    s["v_all"][at // page, :, at % page] = codes[:, 1]
    s["s_all"][at // page, :, at % page] = torch.cat([scales[:, 0], scales[:, 1]], -1)
    return [s["k"], s["v"], s["scales"]]


def _plain_weights(s):
    c, N = s["case"], s["N"]
    B, Hq, Hkv = c["batch"], c["hq"], c["hkv"]
    n = s["seq_lens"].long()[:, None, None]
    pos = torch.arange(N, device=DEV)[None, None]
    last = torch.minimum(pos, n - 1).clamp(min=0)
    k, v = _cached(s, torch.arange(B, device=DEV), last, torch.float32)
    z = (s["q"].float().view(B, Hkv, -1, D) @ k.transpose(2, 3)) * (1 / math.sqrt(D))
    s["logits"].copy_(torch.where(pos < n, z.view(B, Hq, N), s["logits"]))
    e, l = _softmax_parts(z.masked_fill((pos >= n)[:, :, None], -math.inf))
    p = e / torch.where(l > 0, l, 1.0)
    s["out"].copy_((p @ v).view(B, Hq, D))
    w = p.sum(2) + torch.where(pos >= n - c["fresh"], 0.0, s["weights"])
    s["weights"].copy_(torch.where(pos < n, w, s["weights"]))
    return [s["out"], s["weights"], s["logits"]]


def _plain_evict(s):
    c, N, w = s["case"], s["N"], s["weights"]
    B, budget = c["batch"], c["budget"]
    n = s["seq_lens"].long()[:, None, None]
    pos = torch.arange(N, device=DEV)[None, None]
    # kept in any case; then by weight, the lower position first; then what is no token
    key = torch.where((pos < c["sinks"]) | (pos >= n - c["recent"]) | (n <= budget), math.inf, w)
    key = torch.where(pos < n, key, -math.inf)
    best = key.sort(dim=-1, descending=True, stable=True).indices[..., :budget]
    best = torch.where(best < n, best, N).sort(-1).values
    kept = torch.where(best < N, best, -1)
    s["kept"][..., : kept.shape[-1]] = kept
    src = kept.clamp(min=0)
    k, v = _cached(s, torch.arange(B, device=DEV), src, torch.bfloat16)
    moved = w.gather(-1, src)
    b, h, i = torch.nonzero(kept >= 0, as_tuple=True)
    x, page = s["to_k"], s["to_k"].shape[2]
    where = (b, h, i) if s["to_table"] is None else (s["to_table"].long()[b, i // page], h, i % page)
    x[where] = k[b, h, i]
    s["to_v"][where] = v[b, h, i]
    s["to_weights"][b, h, i] = moved[b, h, i]
    s["seq_out"].copy_(s["seq_lens"].clamp(max=budget))
    return [s["kept"], s["to_k"], s["to_v"], s["to_weights"], s["seq_out"]]


def run(s):
    c = s["case"]
    op = c["op"]
    if not own:
        return {"attn": _plain_attn, "append": _plain_append, "weights": _plain_weights,
                "evict": _plain_evict}[op](s)
    import sparse_attention_td_gb300 as td
    if op == "append":
        td.td_q4_append(s["shape"], s["cache"], s["kv_new"][:, 0], s["kv_new"][:, 1], s["slots"])
        # codes and scales as they are held: each is the nearest of its grid, with no room to differ
        return [s["k"], s["v"], s["scales"]]
    if op == "weights":
        td.td_weights_attn(s["shape"], s["cache"], c["fresh"], s["q"], s["seq_lens"], s["weights"],
                           s["logits"], s["out"], ws=s["ws"])
        return [s["out"], s["weights"], s["logits"]]
    if op == "evict":
        td.td_evict(s["shape"], s["cache"], s["to"], c["budget"], c["sinks"], c["recent"], s["weights"],
                    s["to_weights"], s["seq_lens"], s["seq_out"], s["kept"], ws=s["ws"])
        return [s["kept"], s["to_k"], s["to_v"], s["to_weights"], s["seq_out"]]
    if c["k"]:
        td.td_q4_sparse_attn(s["shape"], s["cache"], s["q"], s["seq_lens"], s["idx"], c["k"], s["out"],
                             ws=s["ws"])
        return s["out"]
    call = td.td_q4_attn if c["q4"] else td.td_window_attn
    call(s["shape"], s["cache"], c["window"], c["sinks"], s["cu"] if c["new_hi"] else None, s["q"],
         s["seq_lens"], s["out"], ws=s["ws"])
    return s["out"]


# ---------------------------------------------------------------- 64 bits
def _held(s, which, b, g, rows):
    """Rows of request b and KV head g in 64 bits, one by one from where they are held."""
    x, page, t = s[which], s[which].shape[2], s["table"]
    ids = torch.full_like(rows, b) if t is None else t[b].long()[rows // page]
    at = rows if t is None else rows % page
    if not s["case"].get("q4"):
        return x[ids, g, at].double()
    codes = x[ids, g, at]
    half = torch.stack([codes % 16, codes // 16], -1).flatten(-2).long()
    mag, e = half % 8, (half % 8) // 2
    size = torch.where(e == 0, (mag % 2).double() / 2, (1 + (mag % 2).double() / 2) * 2.0 ** (e - 1).double())
    size = torch.where(half >= 8, -size, size)
    sc = s["scales"][ids, g, at][:, 0 if which == "k" else 8:][:, :8].contiguous()
    return size * sc.view(torch.float8_e4m3fn).double().repeat_interleave(16, -1)


def exact(case, seed):
    """Attention and its weights from their definition in 64 bits, one (request, KV head) at a time.
    The other operators move or code whole values: nothing is computed."""
    if case["op"] not in ("attn", "weights"):
        return None
    s = prepare(case, seed)
    B, Hq, Hkv = case["batch"], case["hq"], case["hkv"]
    G = Hq // Hkv
    weights = case["op"] == "weights"
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    lens = s["seq_lens"].tolist()
    cu = list(range(B + 1)) if weights else s["cu"].tolist()
    if weights:
        w, logits = s["weights"].double(), torch.zeros(B, Hq, s["N"], dtype=torch.float64, device=DEV)
    W = case.get("window", 0)
    for b in range(B):
        n, t = lens[b], cu[b + 1] - cu[b]
        for g in range(Hkv):
            for t0 in range(0, t, 256):
                p = torch.arange(n - t + t0, n - t + min(t, t0 + 256), device=DEV)
                rows = torch.arange(int(p[-1]) + 1, device=DEV)
                if W:
                    rows = rows[(rows < case["sinks"]) | (rows > int(p[0]) - W)]
                if case.get("k"):
                    rows = s["idx"][b, g].long()
                    rows = rows[rows >= 0]
                sees = torch.ones(p.numel(), rows.numel(), dtype=torch.bool, device=DEV)
                if not case.get("k"):
                    gap = p[:, None] - rows[None]
                    sees = gap >= 0
                    if W:
                        sees &= (gap < W) | (rows < case["sinks"])[None]
                at = slice(cu[b] + t0, cu[b] + t0 + p.numel())
                qd = s["q"][at, g * G:(g + 1) * G].double()
                z = torch.einsum("tgd,nd->gtn", qd, _held(s, "k", b, g, rows)) / D ** 0.5
                a = torch.softmax(z.masked_fill(~sees[None], -math.inf), -1)
                out[at, g * G:(g + 1) * G] = torch.einsum("gtn,nd->tgd", a, _held(s, "v", b, g, rows))
                if weights:
                    old = w[b, g, :n].clone()
                    old[max(0, n - case["fresh"]):] = 0
                    w[b, g, :n] = old + a.sum((0, 1))
                    logits[b, g * G:(g + 1) * G, :n] = z[:, 0]
    return [out, w, logits] if weights else out
