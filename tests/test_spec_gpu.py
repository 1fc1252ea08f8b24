"""Speculative-decoding operators on the GPU against plain references."""
import pytest
import torch

import sparse_attention_td_gb300 as td
from spec_util import D, make_mask, pack_mask, paged, reference, tables_reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)


def i32(x):
    return torch.as_tensor(x, dtype=torch.int32).cuda()


def tree_case(seed, G, Hkv, lens, sizes, T, page, kind, k=0, max_len=None):
    """Host inputs: logical rows, everything that holds no token of a request is NaN."""
    gen = torch.Generator().manual_seed(seed)
    B, N = len(lens), max_len or max(max(lens), 1)
    rnd = lambda *s: torch.randn(*s, generator=gen).to(torch.bfloat16)
    c = dict(B=B, G=G, Hkv=Hkv, T=T, N=N, lens=lens, sizes=sizes, page=page, kind=kind)
    c["q"] = 2 * rnd(B, T, G * Hkv, D)
    c["K"], c["V"] = rnd(B, Hkv, N, D), rnd(B, Hkv, N, D)
    for b, n in enumerate(lens):
        c["K"][b, :, n:] = float("nan")
        c["V"][b, :, n:] = float("nan")
    c["seen"] = make_mask(kind, B, T, gen)
    c["idx"] = None
    if k:
        idx = torch.full((B, Hkv, k), -1, dtype=torch.int32)
        for b in range(B):
            ctx = lens[b] - sizes[b]
            for g in range(Hkv):
                n = min(ctx, k - (g % 2))       # rows with and without padding
                idx[b, g, :n] = torch.randperm(max(ctx, 1), generator=gen)[:n].to(torch.int32)
        c["idx"] = idx
    if page:
        blocks = -(-N // page)
        pages = B * blocks + 3
        c["table"] = torch.randperm(pages, generator=gen)[:B * blocks].view(B, blocks).to(torch.int32)
        c["kc"] = paged(c["K"], page, c["table"], pages)
        c["vc"] = paged(c["V"], page, c["table"], pages)
        for b, n in enumerate(lens):            # entries beyond the length are not read
            c["table"][b, -(-n // page):] = 1 << 30
    else:
        c["table"], c["kc"], c["vc"] = None, c["K"], c["V"]
    return c


def run_tree(c, out=None, sizes=True, stream=None, ws=None):
    shape = td.make_shape(c["B"], c["G"] * c["Hkv"], c["Hkv"], c["N"])
    table = None if c["table"] is None else c["table"].cuda()
    cache = td.make_cache(c["kc"].cuda(), c["vc"].cuda(), table)
    q = c["q"].cuda()
    out = torch.full_like(q, 7.0) if out is None else out
    ws = ws or td.Workspace(shape, 0, tree_size=c["T"])
    tl = i32(c["sizes"]) if sizes else None
    mask = None if c["kind"] == "chain" else pack_mask(c["seen"]).cuda()
    if c["idx"] is None:
        td.td_tree_attn(shape, cache, c["T"], tl, mask, q, i32(c["lens"]), out, ws, stream)
    else:
        td.td_tree_sparse_attn(shape, cache, c["T"], tl, mask, q, i32(c["lens"]), c["idx"].cuda(),
                               c["idx"].shape[-1], out, ws, stream)
    torch.cuda.synchronize()
    return out, ws


def check_tree(c, out):
    ref, tol = reference(c["q"], c["K"], c["V"], c["lens"], c["sizes"], c["seen"], c["idx"])
    got = out.cpu().double()
    for b, n in enumerate(c["sizes"]):
        assert torch.all(got[b, n:] == 7.0), f"request {b}: rows behind its tree were written"
        err = (got[b, :n] - ref[b, :n]).abs()
        worst = (err - tol[b, :n]).max().item() if n else 0.0
        assert worst <= 0 and not torch.isnan(err).any(), \
            f"request {b}: error {err.max().item():.3e}, {worst:.3e} over its tolerance"


@pytest.mark.parametrize("page", [0, 16, 64, 128])
@pytest.mark.parametrize("G", [1, 2, 4, 8])
@pytest.mark.parametrize("kind", ["chain", "tree"])
def test_tree_matches_reference(G, page, kind):
    c = tree_case(G * 10 + page, G, 2, [300, 129, 77, 1000], [7, 1, 7, 5], 7, page, kind)
    out, ws = run_tree(c)
    check_tree(c, out)
    assert ws.status() == 0


@pytest.mark.parametrize("T", [1, 2, 16, 31, 33, 64, 100, 128])
@pytest.mark.parametrize("page,k", [(0, 0), (32, 0), (0, 40), (16, 200)])
def test_tree_sizes(T, page, k):
    lens = [T + 300, T, T + 128, T + 3]
    sizes = [T, T, max(1, T - 1), (T + 1) // 2]
    c = tree_case(T + k, 4, 1, lens, sizes, T, page, "tree", k)
    out, ws = run_tree(c)
    check_tree(c, out)
    assert ws.status() == 0


@pytest.mark.parametrize("page", [1, 5, 8, 24, 48, 100, 200, 256, 384])
@pytest.mark.parametrize("k", [0, 60])
def test_any_page_size(page, k):
    c = tree_case(page, 4, 2, [513, 257, 30], [5, 3, 5], 5, page, "tree", k)
    out, ws = run_tree(c)
    check_tree(c, out)
    assert ws.status() == 0


@pytest.mark.parametrize("n", [1, 15, 16, 17, 127, 128, 129, 255, 256, 257, 384, 511])
@pytest.mark.parametrize("page", [0, 16, 128])
def test_context_lengths_around_tiles(n, page):
    c = tree_case(n, 8, 1, [n + 4, n], [4, 1], 4, page, "chain")
    out, ws = run_tree(c)
    check_tree(c, out)
    assert ws.status() == 0


@pytest.mark.parametrize("k", [1, 4, 127, 128, 129, 500])
@pytest.mark.parametrize("page", [0, 16])
def test_sparse_set_sizes(k, page):
    c = tree_case(k, 4, 2, [520, 140, 9], [6, 6, 6], 6, page, "tree", k)
    out, ws = run_tree(c)
    check_tree(c, out)
    assert ws.status() == 0


@pytest.mark.parametrize("kind", ["random", "empty"])
@pytest.mark.parametrize("page", [0, 16])
def test_rows_that_see_nothing_give_zero(kind, page):
    """No context and mask rows without bits: those rows are exactly zero."""
    c = tree_case(3, 4, 2, [9, 200, 9], [9, 9, 4], 9, page, kind)
    c["seen"][0, 2] = False
    out, ws = run_tree(c)
    check_tree(c, out)
    assert torch.all(out[0, 2] == 0)
    assert ws.status() == 0


def test_empty_requests_and_trees():
    c = tree_case(4, 4, 2, [0, 50, 0, 3], [0, 0, 0, 3], 5, 0, "tree", max_len=64)
    out, ws = run_tree(c)
    check_tree(c, out)
    assert ws.status() == 0
    c = tree_case(4, 4, 2, [0, 0], [0, 0], 5, 16, "tree", max_len=64)
    out, _ = run_tree(c)
    assert torch.all(out == 7.0)


def test_tree_lens_may_be_absent():
    c = tree_case(5, 2, 2, [70, 9], [6, 6], 6, 16, "tree")
    out, ws = run_tree(c, sizes=False)
    check_tree(c, out)
    assert ws.status() == 0


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("page,k", [(0, 0), (16, 0), (0, 50)])
def test_values_a_row_does_not_see_never_reach_it(bad, page, k):
    """A drafted token's K and V hold infinities or NaN: rows that see it follow the
    arithmetic (not finite), rows that do not are as if it were absent."""
    c = tree_case(6, 4, 2, [150, 40], [8, 8], 8, page, "random", k)
    c["seen"][:, :, 3] = False
    c["seen"][0, 5, 3] = True
    for what in ("K", "V"):
        cc = dict(c)
        cc[what] = c[what].clone()
        cc[what][0, :, 150 - 8 + 3, 17] = bad
        if page:
            name = {"K": "kc", "V": "vc"}[what]
            cc[name] = c[name].clone()
            p = 150 - 8 + 3
            cc[name][c["table"][0, p // page], :, p % page, 17] = bad
        else:
            cc[{"K": "kc", "V": "vc"}[what]] = cc[what]
        out, ws = run_tree(cc)
        got = out.cpu().double()
        assert not torch.isfinite(got[0, 5]).all() or what == "K"
        if what == "V":
            others = [d for d in range(D) if d != 17]
            assert torch.isfinite(got[0, 5][:, others]).all()
            assert not torch.isfinite(got[0, 5][:, 17]).any()
        ref, tol = reference(c["q"], c["K"], c["V"], c["lens"], c["sizes"], c["seen"], c["idx"])
        for b in range(2):
            rows = [t for t in range(8) if not (b == 0 and t == 5)]
            assert torch.all((got[b, rows] - ref[b, rows]).abs() <= tol[b, rows])
        assert ws.status() == 0


def test_bad_entries_are_skipped_and_reported():
    c = tree_case(7, 4, 2, [100, 90], [4, 4], 4, 16, "chain", 30)
    good = run_tree(c)[0]
    # indexes: beyond the context, below -1; they replace padding, so the result stays
    c2 = dict(c, idx=c["idx"].clone())
    c2["idx"][0, 1, -1] = 96                   # the first drafted position
    c2["idx"][1, 1, -1] = -7
    out, ws = run_tree(c2)
    assert ws.status() == td.FLAG_INDEX_OUT_OF_RANGE
    assert torch.equal(out, good)


@pytest.mark.parametrize("bad", [-1, 1 << 20])
@pytest.mark.parametrize("page", [16, 128, 24])
def test_bad_pages_are_skipped_and_reported(bad, page):
    """A page number outside the cache: its tokens are as if they were absent."""
    c = tree_case(8, 4, 2, [500, 260], [4, 4], 4, page, "chain")
    c["table"][0, 2] = bad
    out, ws = run_tree(c)
    assert ws.status() == td.FLAG_PAGE_OUT_OF_RANGE
    lost = [p for p in range(2 * page, min(3 * page, 500))]
    keep = [p for p in range(500) if p not in lost]
    nt = len([p for p in keep if p >= 496])
    # request 0 without the lost tokens (drafted tokens keep their numbers when none is lost)
    assert nt == 4
    K, V = (c[x].clone() for x in ("K", "V"))
    short = len(keep)
    for x in (K, V):
        x[0, :, :short] = x[0][:, keep]
    ref, tol = reference(c["q"], K, V, [short, 260], c["sizes"], c["seen"])
    assert torch.all((out.cpu().double() - ref).abs() <= tol)


def test_lengths_outside_their_range_are_clamped_and_reported():
    c = tree_case(9, 4, 2, [64, 64], [4, 4], 4, 0, "chain")
    good = run_tree(c)[0]
    out, ws = run_tree(dict(c, lens=[65, 64]))
    assert ws.status() == td.FLAG_SEQ_LEN_OUT_OF_RANGE and torch.equal(out, good)
    out, ws = run_tree(dict(c, sizes=[4, 9]))
    assert ws.status() == td.FLAG_TREE_OUT_OF_RANGE and torch.equal(out, good)
    out, ws = run_tree(dict(c, lens=[-5, 64], sizes=[0, 4]))
    assert ws.status() == td.FLAG_SEQ_LEN_OUT_OF_RANGE
    assert torch.all(out[0] == 7.0) and torch.equal(out[1], good[1])
    out, ws = run_tree(dict(c, lens=[2, 64]))       # four drafted tokens of two
    assert ws.status() == td.FLAG_TREE_OUT_OF_RANGE


def test_one_node_chain_is_plain_decoding():
    """T = 1 over a contiguous cache: td_full_attn_select's output."""
    B, G, Hkv, N = 3, 4, 2, 700
    c = tree_case(10, G, Hkv, [700, 1, 333], [1, 1, 1], 1, 0, "chain")
    out, _ = run_tree(c)
    check_tree(c, out)
    shape = td.make_shape(B, G * Hkv, Hkv, N)
    ws = td.Workspace(shape, 0)
    q = c["q"].cuda().view(B, G * Hkv, D)
    ref = torch.empty_like(q)
    td.td_full_attn_select(shape, q, c["kc"].nan_to_num().cuda(), c["vc"].nan_to_num().cuda(),
                           i32(c["lens"]), 0, None, ref, ws=ws)
    torch.cuda.synchronize()
    # both within the tolerance of the 64-bit result
    r, tol = reference(c["q"], c["K"], c["V"], c["lens"], c["sizes"], c["seen"])
    assert torch.all((ref.cpu().double() - r[:, 0]).abs() <= tol[:, 0])


def test_results_do_not_change_from_call_to_call_or_stream_to_stream():
    a = tree_case(11, 4, 2, [2500, 900, 40], [16, 16, 9], 16, 64, "tree")
    b = tree_case(12, 8, 1, [4000, 17], [30, 4], 30, 0, "tree")
    wa, wb = (td.Workspace(td.make_shape(c["B"], c["G"] * c["Hkv"], c["Hkv"], c["N"]), 0,
                           tree_size=c["T"]) for c in (a, b))
    ra, rb = run_tree(a, ws=wa)[0], run_tree(b, ws=wb)[0]
    check_tree(a, ra)
    check_tree(b, rb)
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()

    def device(c, ws):
        shape = td.make_shape(c["B"], c["G"] * c["Hkv"], c["Hkv"], c["N"])
        table = None if c["table"] is None else c["table"].cuda()
        q = c["q"].cuda()
        return (shape, td.make_cache(c["kc"].cuda(), c["vc"].cuda(), table), c["T"], i32(c["sizes"]),
                pack_mask(c["seen"]).cuda(), q, i32(c["lens"])), torch.full_like(q, 7.0), ws

    (xa, oa, wa), (xb, ob, wb) = device(a, wa), device(b, wb)
    torch.cuda.synchronize()
    for _ in range(5):
        oa.fill_(7.0), ob.fill_(7.0)
        torch.cuda.synchronize()
        for _ in range(4):
            td.td_tree_attn(*xa, oa, wa, stream=sa)
            td.td_tree_attn(*xb, ob, wb, stream=sb)
        torch.cuda.synchronize()
        assert torch.equal(oa, ra) and torch.equal(ob, rb)


def test_captured_call_follows_its_buffers():
    c = tree_case(13, 4, 2, [600, 300], [8, 8], 8, 16, "tree")
    shape = td.make_shape(2, 8, 2, 600)
    cache = td.make_cache(c["kc"].cuda(), c["vc"].cuda(), c["table"].cuda())
    q, lens, sizes = c["q"].cuda(), i32(c["lens"]), i32(c["sizes"])
    mask, ws = pack_mask(c["seen"]).cuda(), td.Workspace(shape, 0, tree_size=8)
    out = torch.full_like(q, 7.0)
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        td.td_tree_attn(shape, cache, 8, sizes, mask, q, lens, out, ws)
    g.replay()
    torch.cuda.synchronize()
    check_tree(c, out)
    c2 = dict(c, lens=[411, 90], sizes=[3, 8])
    c2["K"], c2["V"] = c["K"], c["V"]
    lens.copy_(i32(c2["lens"])), sizes.copy_(i32(c2["sizes"]))
    out.fill_(7.0)
    g.replay()
    torch.cuda.synchronize()
    check_tree(c2, out)
    assert ws.status() == 0


# ------------------------------------------------------------- moves of rows
def test_append_slots():
    gen = torch.Generator().manual_seed(1)
    pages, Hkv, page = 9, 3, 16
    for n in (1, 7, 100):
        k = torch.randn(pages, Hkv, page, D, generator=gen).to(torch.bfloat16)
        v = torch.randn(pages, Hkv, page, D, generator=gen).to(torch.bfloat16)
        new = torch.randn(n, 5 * Hkv, D, generator=gen).to(torch.bfloat16)   # q, k, v of a packed projection
        slots = torch.randperm(pages * page, generator=gen)[:n].to(torch.int32)
        slots[n // 2] = [-1, pages * page, 1 << 30][n % 3]
        kd, vd, nd = k.cuda(), v.cuda(), new.cuda()
        shape = td.make_shape(1, Hkv, Hkv, pages * page)
        td.td_kv_append_slots(shape, td.make_cache(kd, vd), nd[:, 3 * Hkv:4 * Hkv],
                              nd[:, 4 * Hkv:], slots.cuda())
        torch.cuda.synchronize()
        for i, s in enumerate(slots.tolist()):
            if 0 <= s < pages * page:
                k[s // page, :, s % page] = new[i, 3 * Hkv:4 * Hkv]
                v[s // page, :, s % page] = new[i, 4 * Hkv:]
        assert torch.equal(kd.cpu(), k) and torch.equal(vd.cpu(), v)


def test_append_slots_refuses_other_layouts():
    k = torch.zeros(4, 2, 16, D, dtype=torch.bfloat16, device="cuda")
    cache, shape = td.make_cache(k, k.clone()), td.make_shape(1, 2, 2, 64)
    x = torch.zeros(3, 2, D, dtype=torch.bfloat16, device="cuda")
    slots = i32([0, 1, 2])
    with pytest.raises(ValueError):
        td.td_kv_append_slots(shape, cache, x.transpose(0, 1), x, slots)
    with pytest.raises(ValueError):
        td.td_kv_append_slots(shape, cache, x.float(), x, slots)
    with pytest.raises(ValueError):
        td.td_kv_append_slots(shape, cache, x, x[:2], slots)
    with pytest.raises(ValueError):
        td.td_kv_append_slots(shape, cache, x, x, slots[:2])
    with pytest.raises(ValueError):
        td.td_kv_append_slots(td.make_shape(1, 4, 4, 64), cache, x, x, slots)
    with pytest.raises(ValueError):
        td.make_cache(k.cpu(), k)
    with pytest.raises(ValueError):
        td.make_cache(k[:, :, :8], k[:, :, :8])
    with pytest.raises(ValueError):
        td.make_cache(k, k, torch.zeros(4, 4, dtype=torch.int64, device="cuda"))


@pytest.mark.parametrize("page", [0, 16, 24])
@pytest.mark.parametrize("layers", [1, 3, 33])
def test_commit_moves_the_accepted_rows(page, layers):
    gen = torch.Generator().manual_seed(layers + page)
    B, Hkv, T, N = 4, 2, 40, 100
    lens, sizes = [100, 60, 40, 33], [40, 20, 40, 33]
    acc = [torch.randperm(40, generator=gen)[:17].sort().values.tolist(),      # a path
           [1, 0, 0, 19, 2],                                                   # any order, repeated
           list(range(1, 40)),                                                 # every row moves by one
           []]
    accepted = torch.full((B, T), -5, dtype=torch.int32)
    for b, a in enumerate(acc):
        accepted[b, :len(a)] = torch.tensor(a, dtype=torch.int32)
    table = None
    blocks = -(-N // page) if page else 1
    dims = (B * blocks, Hkv, page, D) if page else (B, Hkv, N, D)
    if page:
        table = torch.randperm(B * blocks, generator=gen).view(B, blocks).to(torch.int32)
    ks = [torch.randn(dims, generator=gen).to(torch.bfloat16) for _ in range(layers)]
    vs = [torch.randn(dims, generator=gen).to(torch.bfloat16) for _ in range(layers)]
    kd, vd = [x.cuda() for x in ks], [x.cuda() for x in vs]
    td_table = None if table is None else table.cuda()
    shape = td.make_shape(B, Hkv, Hkv, N)
    ws = td.Workspace(shape, 0)
    out = torch.full((B,), -9, dtype=torch.int32, device="cuda")
    td.td_tree_commit(shape, [td.make_cache(a, b, td_table) for a, b in zip(kd, vd)], T, i32(sizes),
                      accepted.cuda(), i32([len(a) for a in acc]), i32(lens), out, ws)
    torch.cuda.synchronize()
    assert out.tolist() == [lens[b] - sizes[b] + len(acc[b]) for b in range(B)]
    for x in ks + vs:
        old = x.clone()
        for b, a in enumerate(acc):
            ctx = lens[b] - sizes[b]
            at = (lambda p: (table[b, p // page], p % page)) if page else (lambda p: (b, p))
            for i, j in enumerate(a):
                (pd, rd), (ps, rs) = at(ctx + i), at(ctx + j)
                x[pd, :, rd] = old[ps, :, rs]
    for got, ref in zip(kd + vd, ks + vs):
        assert torch.equal(got.cpu(), ref)
    assert ws.status() == 0


def test_commit_reports_bad_nodes():
    k = torch.randn(1, 1, 20, D).to(torch.bfloat16).cuda()
    v = k.clone()
    old = k.clone()
    shape = td.make_shape(1, 1, 1, 20)
    ws = td.Workspace(shape, 0)
    out = torch.zeros(1, dtype=torch.int32, device="cuda")
    td.td_tree_commit(shape, [td.make_cache(k, v)], 6, i32([6]), i32([2, 6, -1, 5, 0, 0]), i32([4]),
                      i32([20]), out, ws)
    torch.cuda.synchronize()
    assert ws.status() == td.FLAG_TREE_OUT_OF_RANGE and out.item() == 18
    old[0, :, 14], old[0, :, 17] = old[0, :, 16].clone(), old[0, :, 19].clone()
    assert torch.equal(k, old) and torch.equal(v, old)
    td.td_tree_commit(shape, [td.make_cache(k, v)], 6, i32([6]), i32([0] * 6), i32([9]), i32([20]),
                      out, ws)
    torch.cuda.synchronize()
    assert ws.status() == td.FLAG_TREE_OUT_OF_RANGE and out.item() == 20


# --------------------------------------------------------------- block tables
def run_tables(page, blocks, pages, lens, new, table, held, free, count, max_new, in_place=False):
    t, h, f, c = i32(table), i32(held), i32(free), i32([count])
    ho = h if in_place else torch.full_like(h, -9)
    co = c if in_place else torch.full_like(c, -9)
    cu = torch.full((len(lens) + 1,), -9, dtype=torch.int32, device="cuda")
    slots = torch.full((max_new,), -9, dtype=torch.int32, device="cuda")
    ws = td.Workspace(td.make_shape(1, 1, 1, 1), 0)
    for _ in range(1 if in_place else 2):      # separate outputs: the call can be repeated
        td.td_block_tables(i32(lens), i32(new), page, t, h, ho, f, c, co, cu, slots, ws)
    torch.cuda.synchronize()
    return t, ho, f, co, cu, slots, ws.status()


def check_tables(page, blocks, pages, lens, new, table, held, free, count, max_new, flags=0):
    ref = tables_reference(page, blocks, pages, lens, new, table, held, free, count, max_new)
    for in_place in (False, True):
        t, h, f, c, cu, slots, st = run_tables(page, blocks, pages, lens, new, table, held, free,
                                               count, max_new, in_place)
        assert t.tolist() == ref[0]
        assert h.tolist() == ref[1]
        assert c.item() == len(ref[2]) and f.tolist()[:c.item()] == ref[2]
        assert cu.tolist() == ref[3]
        assert slots.tolist() == ref[4]
        assert st == flags | (td.FLAG_PAGES_EXHAUSTED if ref[5] else 0)
    return ref


def tables_case(seed, B, page, hi, spare, shrink=0.2, grow=False):
    """Requests that grow, shrink, finish and start (grow: none gives a page back), with `spare`
    free pages beyond what they need."""
    gen = torch.Generator().manual_seed(seed)
    r = lambda n, *s: torch.randint(0, n, s, generator=gen)
    lens, old = r(hi + 1, B), r(hi + 1, B)
    lens = torch.where(torch.rand(B, generator=gen) < shrink, torch.minimum(lens, old), lens)
    old = torch.minimum(old, lens) if grow else old
    new = torch.minimum(lens, r(40, B))
    held = (old + page - 1) // page
    blocks = -(-hi // page)
    need = ((lens + page - 1) // page - held).clamp(min=0).sum().item()
    back = (held - (lens + page - 1) // page).clamp(min=0).sum().item()
    count = max(0, need - back + spare)
    pages = int(held.sum()) + count + 5
    ids = torch.randperm(pages, generator=gen).tolist()
    table = [[-1] * blocks for _ in range(B)]
    for b in range(B):
        for j in range(int(held[b])):
            table[b][j] = ids.pop()
    free = ids[:count] + [-1] * (pages - count)
    return (page, blocks, pages, lens.tolist(), new.tolist(), table, held.tolist(), free, count)


@pytest.mark.parametrize("B", [1, 2, 33, 257, 1024, 1025, 2600])
@pytest.mark.parametrize("page", [1, 16, 30, 64])
def test_block_tables_match_reference(B, page):
    a = tables_case(B + page, B, page, 200 if B > 300 else 700, 3)
    check_tables(*a, max_new=sum(a[4]) + 11)


@pytest.mark.parametrize("short", [1, 7, 60])
@pytest.mark.parametrize("B", [9, 1500])
def test_block_tables_run_out_of_pages(B, short):
    a = tables_case(short, B, 16, 600, -short, shrink=0.0, grow=True)
    ref = check_tables(*a, max_new=sum(a[4]) + 3)
    assert ref[5]


def test_block_tables_slot_map_too_short_or_empty():
    a = tables_case(2, 20, 16, 300, 4)
    assert check_tables(*a, max_new=sum(a[4]) - 5)[5]
    assert check_tables(*a, max_new=0)[5]
    page, blocks, pages, lens, new, table, held, free, count = a
    check_tables(page, blocks, pages, lens, [0] * len(lens), table, held, free, count, max_new=4)


def test_block_tables_everything_is_released():
    page, blocks, pages, lens, new, table, held, free, count = tables_case(3, 50, 16, 300, 4)
    ref = check_tables(page, blocks, pages, [0] * 50, [0] * 50, table, held, free, count, max_new=1)
    assert ref[1] == [0] * 50 and len(ref[2]) == sum(held) + count


def test_block_tables_report_bad_input():
    lens, new = [500, -3, 20], [4, 2, 30]
    table, held = [[0, 1, -1, -1], [2, -1, -1, -1], [3, -1, -1, -1]], [2, 9, 1]
    free, count = [4, 5, 99, 7, 8, 9, 10, 11] + [-1] * 8, 8
    t, h, f, c, cu, slots, st = run_tables(16, 4, 16, lens, new, table, held, free, count, 40)
    assert st == td.FLAG_SEQ_LEN_OUT_OF_RANGE | td.FLAG_PAGE_OUT_OF_RANGE
    assert h.tolist() == [4, 0, 2] and cu.tolist() == [0, 4, 4, 24]
    # request 1 gave back its page 2 and three entries that hold no page; those came out first
    assert t.tolist() == [[0, 1, -1, -1], [2, -1, -1, -1], [3, -1, -1, -1]]
    assert c.item() == 9 and f[:9].tolist() == [4, 5, 99, 7, 8, 9, 10, 11, 2]
    assert slots.tolist() == [-1] * 4 + list(range(48, 64)) + [-1] * 20
    # a page number outside the pool is handed out as it is, and gives no slots
    t, h, f, c, cu, slots, st = run_tables(16, 4, 16, [10], [10], [[-1] * 4], [0], [99] + [-1] * 15,
                                           1, 12)
    assert st == td.FLAG_PAGE_OUT_OF_RANGE and slots.tolist() == [-1] * 12
    # a stack count outside the pool
    for count, want in ((-4, 0), (17, 16)):
        *_, c, cu, slots, st = run_tables(16, 4, 16, [0], [0], [[-1] * 4], [0], list(range(16)), count, 2)
        assert st == td.FLAG_PAGE_OUT_OF_RANGE and c.item() == want


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("sparse", [False, True])
def test_speculative_steps_on_pages(sparse, captured):
    """Three speculative steps of a ragged batch: tables, append, attention, commit; the
    cache, the lengths and the outputs follow a plain simulation of the sequences."""
    gen = torch.Generator().manual_seed(21)
    B, G, Hkv, T, page, N, layers, k = 3, 4, 2, 6, 16, 160, 2, 24
    rnd = lambda *s: torch.randn(*s, generator=gen).to(torch.bfloat16)
    blocks, pages = N // page, 40
    shape = td.make_shape(B, G * Hkv, Hkv, N)
    ws = td.Workspace(shape, 0, tree_size=T)
    nan = lambda: torch.full((pages, Hkv, page, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    table = torch.full((B, blocks), -1, dtype=torch.int32, device="cuda")
    caches = [td.make_cache(nan(), nan(), table) for _ in range(layers)]
    held, held2 = i32([0] * B), i32([0] * B)
    free, count, count2 = torch.randperm(pages, generator=gen).to(torch.int32).cuda(), i32([pages]), i32([0])
    cu = i32([0] * (B + 1))
    ctx = [33, 1, 90]
    K, V = (rnd(layers, B, Hkv, N, D) for _ in range(2))          # the sequences as they should be
    sizes = [6, 4, 5]
    # the prompts
    lens = i32(ctx)
    slots = torch.zeros(sum(ctx) + 5, dtype=torch.int32, device="cuda")
    td.td_block_tables(lens, lens.clone(), page, table, held, held, free, count, count, cu, slots, ws)
    pad = torch.zeros(5, Hkv, D, dtype=torch.bfloat16)
    for l in range(layers):
        kn, vn = (torch.cat([x[l, b, :, :ctx[b]].transpose(0, 1) for b in range(B)] + [pad])
                  for x in (K, V))
        td.td_kv_append_slots(shape, caches[l], kn.cuda(), vn.cuda(), slots)
    # static buffers of a step
    seq, tl, acc, al = i32([0] * B), i32(sizes), i32([[0] * T] * B), i32([0] * B)
    new_seq = i32([0] * B)
    kvn = torch.zeros(layers, B * T, 2, Hkv, D, dtype=torch.bfloat16, device="cuda")
    q = torch.zeros(layers, B, T, G * Hkv, D, dtype=torch.bfloat16, device="cuda")
    out = torch.full_like(q, 7.0)
    mask = torch.zeros(B, T, 1, dtype=torch.int32, device="cuda")
    idx = torch.zeros(B, Hkv, k, dtype=torch.int32, device="cuda")
    step_slots = torch.zeros(B * T, dtype=torch.int32, device="cuda")

    def attend():
        td.td_block_tables(seq, tl, page, table, held, held2, free, count, count2, cu, step_slots, ws)
        for l in range(layers):
            td.td_kv_append_slots(shape, caches[l], kvn[l, :, 0], kvn[l, :, 1], step_slots)
            if sparse:
                td.td_tree_sparse_attn(shape, caches[l], T, tl, mask, q[l], seq, idx, k, out[l], ws)
            else:
                td.td_tree_attn(shape, caches[l], T, tl, mask, q[l], seq, out[l], ws)

    def commit():
        td.td_tree_commit(shape, caches, T, tl, acc, al, seq, new_seq, ws)

    graphs = None
    if captured:
        graphs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]
        torch.cuda.synchronize()
        for g, f in zip(graphs, (attend, commit)):
            with torch.cuda.graph(g):
                f()
    for step in range(3):
        lens_now = [c + s for c, s in zip(ctx, sizes)]
        seen = make_mask("tree", B, T, gen)
        draft = rnd(layers, B, T, 2, Hkv, D)
        qs = 2 * rnd(layers, B, T, G * Hkv, D)
        ids = torch.full((B, Hkv, k), -1, dtype=torch.int32)
        for b in range(B):
            for g in range(Hkv):
                n = min(k, ctx[b])
                ids[b, g, :n] = torch.randperm(ctx[b], generator=gen)[:n].sort().values.to(torch.int32)
        packed = torch.zeros_like(kvn, device="cpu")
        at = 0
        for b in range(B):
            for j in range(sizes[b]):
                packed[:, at] = draft[:, b, j]
                K[:, b, :, ctx[b] + j], V[:, b, :, ctx[b] + j] = draft[:, b, j, 0], draft[:, b, j, 1]
                at += 1
        for dst, src in ((seq, i32(lens_now)), (kvn, packed), (q, qs), (mask, pack_mask(seen)), (idx, ids)):
            dst.copy_(src)
        out.fill_(7.0)
        graphs[0].replay() if captured else attend()
        held.copy_(held2), count.copy_(count2)
        torch.cuda.synchronize()
        for l in range(layers):
            c = dict(q=qs[l], K=K[l], V=V[l], lens=lens_now, sizes=sizes, seen=seen,
                     idx=ids if sparse else None)
            check_tree(c, out[l])
        kept = []
        for b in range(B):
            path = [j for j in range(sizes[b]) if seen[b, sizes[b] - 1, j]][:1 + (step + b) % 4]
            kept.append(path)
            for x in (K, V):
                x[:, b, :, ctx[b]:ctx[b] + len(path)] = x[:, b][:, :, [ctx[b] + j for j in path]]
        a = torch.zeros(B, T, dtype=torch.int32)
        for b, p in enumerate(kept):
            a[b, :len(p)] = torch.tensor(p, dtype=torch.int32)
        acc.copy_(a), al.copy_(i32([len(p) for p in kept]))
        graphs[1].replay() if captured else commit()
        torch.cuda.synchronize()
        ctx = [c + len(p) for c, p in zip(ctx, kept)]
        assert new_seq.tolist() == ctx
        assert ws.status() == 0
        t = table.cpu()
        for l in range(layers):
            for x, ref in ((caches[l].k.cpu(), K[l]), (caches[l].v.cpu(), V[l])):
                for b in range(B):
                    pos = torch.arange(ctx[b])
                    got = x[t[b, pos // page].long(), :, pos % page]
                    assert torch.equal(got, ref[b, :, :ctx[b]].transpose(0, 1))
    # the pages all come back
    td.td_block_tables(i32([0] * B), i32([0] * B), page, table, held, held, free, count, count, cu,
                       step_slots, ws)
    torch.cuda.synchronize()
    assert count.item() == pages and sorted(free.tolist()) == list(range(pages))


def test_selection_then_tree_layers_on_a_contiguous_cache():
    """A selection layer's set (from the last accepted token's query) serves the sparse tree
    layers of the same step."""
    B, G, Hkv, T, N, k = 2, 4, 2, 5, 900, 64
    c = tree_case(31, G, Hkv, [900, 500], [5, 5], T, 0, "chain")
    for x in ("K", "V"):
        c[x] = c[x].nan_to_num()
    c["kc"], c["vc"] = c["K"], c["V"]
    shape = td.make_shape(B, G * Hkv, Hkv, N)
    ws = td.Workspace(shape, k, tree_size=T)        # one buffer for both kinds of calls
    K, V, q = c["kc"].cuda(), c["vc"].cuda(), c["q"].cuda()
    idx = torch.full((B, Hkv, k), -1, dtype=torch.int32, device="cuda")
    root = torch.empty(B, G * Hkv, D, dtype=torch.bfloat16, device="cuda")
    ctx = i32([895, 495])
    out = torch.full_like(q, 7.0)
    sets = []
    for _ in range(2):
        td.td_full_attn_select(shape, q[:, 0].contiguous(), K, V, ctx, k, idx, root, ws=ws)
        td.td_tree_sparse_attn(shape, td.make_cache(K, V), T, i32([5, 5]), None, q, i32(c["lens"]),
                               idx, k, out, ws)
        torch.cuda.synchronize()
        sets.append((idx.cpu(), root.cpu()))
        c["idx"] = idx.cpu()
        check_tree(c, out)
    assert torch.equal(sets[0][0], sets[1][0]) and torch.equal(sets[0][1], sets[1][1])
    assert ws.status() == 0


def test_tensors_of_the_wrong_size_are_refused():
    c = tree_case(14, 4, 2, [60, 30], [4, 4], 4, 16, "tree")
    shape = td.make_shape(2, 8, 2, 60)
    cache = td.make_cache(c["kc"].cuda(), c["vc"].cuda(), c["table"].cuda())
    q, lens, ws = c["q"].cuda(), i32(c["lens"]), td.Workspace(shape, 0, tree_size=4)
    mask, out = pack_mask(c["seen"]).cuda(), torch.empty_like(q)
    call = lambda **kw: td.td_tree_attn(*({**dict(
        shape=shape, cache=cache, tree_size=4, tree_lens=None, tree_mask=mask, q=q, seq_lens=lens,
        out=out, ws=ws), **kw}.values()))
    call()
    for kw in (dict(q=q[:1]), dict(q=q.float()), dict(q=q.cpu()), dict(seq_lens=lens[:1]),
               dict(out=out[:, :3].contiguous()), dict(tree_mask=mask[:1]),
               dict(seq_lens=lens.long()), dict(q=q.transpose(1, 2)),
               dict(shape=td.make_shape(3, 8, 2, 60)), dict(shape=td.make_shape(2, 8, 4, 60))):
        with pytest.raises(ValueError):
            call(**kw)
    with pytest.raises(td.TdError):
        call(tree_size=0)
    with pytest.raises(td.TdError):
        call(shape=td.make_shape(2, 8, 2, 100))       # more positions than the tables hold
    torch.cuda.synchronize()
