"""Tree attention where its work is cut unevenly: many small requests, few long
ones, several blocks of query rows, and drafted tokens around a tile's end."""
import pytest
import torch

import sparse_attention_td_gb300 as td
from spec_util import D
from test_spec_gpu import _built, check_tree, run_tree, tree_case  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("page", [0, 16])
@pytest.mark.parametrize("k", [0, 20])
def test_many_small_requests(page, k):
    """More requests than threads in a block, many units per SM, some without work."""
    gen = torch.Generator().manual_seed(page + k)
    B = 700
    lens = torch.randint(0, 60, (B,), generator=gen).tolist()
    sizes = [min(n, int(s)) for n, s in zip(lens, torch.randint(0, 4, (B,), generator=gen))]
    c = tree_case(page + k, 2, 1, lens, sizes, 3, page, "tree", k, max_len=64)
    out, ws = run_tree(c)
    check_tree(c, out)
    assert ws.status() == 0


@pytest.mark.parametrize("page", [0, 64])
@pytest.mark.parametrize("G,T", [(1, 2), (8, 3), (8, 20)])
def test_one_long_request_on_every_sm(page, G, T):
    """One (request, KV head) in parts on all SMs."""
    c = tree_case(G, G, 1, [40003], [T], T, page, "tree")
    out, ws = run_tree(c)
    check_tree(c, out)
    assert ws.status() == 0
    assert torch.equal(run_tree(c)[0], out)


@pytest.mark.parametrize("ctx", [1, 63, 64, 65, 100, 120, 126, 127, 128, 129, 200, 256])
@pytest.mark.parametrize("nt", [1, 2, 8, 28, 64, 65, 127, 128])
def test_drafted_tokens_around_a_tiles_end(ctx, nt):
    """Sharing the last context tile, just fitting it, or in one of their own."""
    c = tree_case(ctx * 131 + nt, 1, 1, [ctx + nt], [nt], 128, 32, "random")
    c["seen"][0, :, 0] = True
    out, ws = run_tree(c)
    check_tree(c, out)
    assert ws.status() == 0


@pytest.mark.parametrize("G,T", [(4, 64), (8, 64), (8, 128), (2, 100), (1, 128)])
@pytest.mark.parametrize("page,k", [(0, 0), (16, 0), (128, 0), (0, 150), (16, 150)])
def test_blocks_of_query_rows(G, T, page, k):
    """Over 128 rows per KV head: several blocks of rows; requests whose trees fill one block
    only lie between them."""
    lens = [T + 400, 5, T + 131, 40, T + 7]
    sizes = [T, 3, T - 1, min(T, 17), T // 2 + 1]
    c = tree_case(G * T + page + k, G, 1, lens, sizes, T, page, "tree", k)
    out, ws = run_tree(c)
    check_tree(c, out)
    assert ws.status() == 0


@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
@pytest.mark.parametrize("ctx", [0, 70, 256])
def test_non_finite_values_with_two_row_tiles(bad, ctx):
    T, G = 50, 4
    c = tree_case(ctx, G, 1, [ctx + T, ctx + T], [T, T], T, 0, "random")
    c["seen"][0, :, 7] = False
    c["seen"][0, (3, 40), 7] = True            # a row of each row tile sees the token
    cc = dict(c, V=c["V"].clone())
    cc["V"][0, 0, ctx + 7, 100] = bad
    cc["vc"] = cc["V"]
    out, ws = run_tree(cc)
    clean, _ = run_tree(c)
    check_tree(c, clean)
    got = out.cpu()
    for t in (3, 40):
        assert not torch.isfinite(got[0, t, :, 100]).any()
        other = [d for d in range(D) if d != 100]
        assert torch.equal(got[0, t][:, other], clean[0, t].cpu()[:, other])
    rows = [t for t in range(T) if t not in (3, 40)]
    assert torch.equal(got[0, rows], clean[0, rows].cpu()) and torch.equal(got[1], clean[1].cpu())
    assert ws.status() == 0


@pytest.mark.parametrize("page", [16, 24])
def test_bad_pages_of_a_sparse_layer(page):
    """Index entries on a page outside the cache count as absent."""
    c = tree_case(5, 4, 2, [300, 200], [6, 6], 6, page, "chain", 40)
    c["table"][0, 3] = -4
    out, ws = run_tree(c)
    assert ws.status() == td.FLAG_PAGE_OUT_OF_RANGE
    gone = dict(c, idx=c["idx"].clone())
    hit = (gone["idx"][0] >= 3 * page) & (gone["idx"][0] < 4 * page)
    gone["idx"][0][hit] = -1
    assert hit.any()
    check_tree(gone, out)


def test_two_captured_graphs_share_a_workspace():
    """Replayed one after the other on one stream, in any order."""
    a = tree_case(1, 4, 2, [3000, 1500], [8, 5], 8, 16, "tree")
    b = tree_case(2, 4, 2, [700, 2600], [40, 33], 40, 0, "tree", 300)
    from test_spec_gpu import i32
    from spec_util import pack_mask
    shape = [td.make_shape(2, 8, 2, c["N"]) for c in (a, b)]
    big = max(shape, key=lambda s: td.td_tree_workspace_size(s, 40))
    ws = td.Workspace(big, 0, tree_size=40)
    graphs, outs, keep = [], [], []
    for c, s in zip((a, b), shape):
        table = None if c["table"] is None else c["table"].cuda()
        x = dict(cache=td.make_cache(c["kc"].cuda(), c["vc"].cuda(), table), q=c["q"].cuda(),
                 mask=pack_mask(c["seen"]).cuda(), lens=i32(c["lens"]), sizes=i32(c["sizes"]),
                 idx=None if c["idx"] is None else c["idx"].cuda())
        x["out"] = torch.full_like(x["q"], 7.0)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            if x["idx"] is None:
                td.td_tree_attn(s, x["cache"], c["T"], x["sizes"], x["mask"], x["q"], x["lens"], x["out"], ws)
            else:
                td.td_tree_sparse_attn(s, x["cache"], c["T"], x["sizes"], x["mask"], x["q"], x["lens"],
                                       x["idx"], c["idx"].shape[-1], x["out"], ws)
        graphs.append(g), outs.append(x["out"]), keep.append(x)
    for order in ((0, 1), (1, 0), (0, 0, 1, 1, 0)):
        for o in outs:
            o.fill_(7.0)
        for i in order:
            graphs[i].replay()
        torch.cuda.synchronize()
        check_tree(a, outs[0])
        check_tree(b, outs[1])
    assert ws.status() == 0


@pytest.mark.parametrize("page,k", [(0, 0), (16, 0), (16, 40)])
def test_small_and_large_trees_in_turn(page, k):
    """Two blocks of rows in some requests, most with rows for one only and one tile of tokens."""
    gen = torch.Generator().manual_seed(page + k)
    B, T = 220, 40
    sizes = [40 if b % 7 == 3 else int(s) for b, s in enumerate(torch.randint(0, 20, (B,), generator=gen))]
    lens = [n + int(c) for n, c in zip(sizes, torch.randint(0, 150, (B,), generator=gen))]
    c = tree_case(page + k, 4, 2, lens, sizes, T, page, "tree", k, max_len=192)
    out, ws = run_tree(c)
    check_tree(c, out)
    assert ws.status() == 0
    assert torch.equal(run_tree(c)[0], out)


def test_non_finite_values_of_neighbouring_units():
    """One-tile units, every second one with values that are not finite in its tree: they stay
    with the rows that see them and with their unit."""
    B, T, page = 400, 4, 16
    gen = torch.Generator().manual_seed(5)
    lens = (T + torch.randint(0, 100, (B,), generator=gen)).tolist()
    c = tree_case(9, 2, 2, lens, [T] * B, T, page, "tree", max_len=112)
    c["seen"][:, :, 2] = False
    c["seen"][:, 3, 2] = True                     # only the last row sees token 2
    for b in range(0, B, 2):
        p = lens[b] - T + 2
        c["vc"][c["table"][b, p // page], :, p % page, 5] = float("inf")
        c["V"][b, :, p, 5] = 0.0                  # what the rows that do not see it get is unchanged
    out, ws = run_tree(c)
    hit = torch.zeros_like(out, dtype=torch.bool)
    hit[0::2, 3, :, 5] = True
    assert torch.all(out[hit] == float("inf"))
    out[hit] = 0.0
    from spec_util import reference
    ref, tol = reference(c["q"], c["K"], c["V"], c["lens"], c["sizes"], c["seen"])
    ref[0::2, 3, :, 5] = 0.0
    err = (out.cpu().double() - ref).abs()
    assert torch.all(err <= tol) and ws.status() == 0


def test_rows_behind_32_bit_offsets():
    """A cache of more than 2^32 bytes and values: pages, slots and committed rows at its end."""
    B, Hkv, G, page, T = 2, 8, 1, 64, 5
    pages = (1 << 32) // (Hkv * page * D) + 64           # values per tensor over 2^32
    c = tree_case(21, G, Hkv, [300, 130], [T, T], T, page, "tree")
    blocks = c["table"].shape[1]
    table = torch.arange(pages - 2 * blocks, pages, dtype=torch.int32).view(2, blocks)
    shape = td.make_shape(B, Hkv * G, Hkv, c["N"])
    kc = torch.empty(pages, Hkv, page, D, dtype=torch.bfloat16, device="cuda")
    vc = torch.empty_like(kc)
    cache = td.make_cache(kc, vc, table.cuda())
    ws = td.Workspace(shape, 0, tree_size=T)
    pos = [(b, p) for b in range(B) for p in range(c["lens"][b])]
    slots = torch.tensor([int(table[b, p // page]) * page + p % page for b, p in pos], dtype=torch.int32)
    new = [torch.stack([x[b, :, p] for b, p in pos]).cuda() for x in (c["K"], c["V"])]
    td.td_kv_append_slots(shape, cache, new[0], new[1], slots.cuda())
    q, out = c["q"].cuda(), torch.full_like(c["q"], 7.0).cuda()
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    from spec_util import pack_mask
    td.td_tree_attn(shape, cache, T, None, pack_mask(c["seen"]).cuda(), q, i32(c["lens"]), out, ws)
    torch.cuda.synchronize()
    check_tree(c, out)
    kept = [0, 2, 4]
    new_lens = i32([0, 0])
    td.td_tree_commit(shape, [cache], T, None, i32([kept + [0, 0]] * B), i32([3] * B), i32(c["lens"]), new_lens, ws)
    torch.cuda.synchronize()
    assert new_lens.tolist() == [n - T + 3 for n in c["lens"]] and ws.status() == 0
    for b, n in enumerate(c["lens"]):
        for i, j in enumerate(kept):
            at, src = n - T + i, n - T + j
            for got, x in ((kc, c["K"]), (vc, c["V"])):
                assert torch.equal(got[int(table[b, at // page]), :, at % page].cpu(), x[b, :, src])
    del kc, vc, cache
    torch.cuda.empty_cache()


def test_captured_behind_other_work():
    """The calls of a step captured behind a fill, a copy and another stream's work, each of which
    writes what the call reads."""
    from test_spec_gpu import i32
    from spec_util import pack_mask
    c = tree_case(31, 4, 2, [900, 333], [8, 5], 8, 16, "tree")
    shape = td.make_shape(2, 8, 2, c["N"])
    ws = td.Workspace(shape, 0, tree_size=8)
    pages, _, page, _ = c["kc"].shape
    rows = [x.permute(0, 2, 1, 3).reshape(pages * page, 2, D).contiguous().cuda() for x in (c["kc"], c["vc"])]
    k, v = torch.zeros_like(c["kc"]).cuda(), torch.zeros_like(c["vc"]).cuda()
    cache = td.make_cache(k, v, c["table"].cuda())
    slots = torch.full((pages * page,), -1, dtype=torch.int32, device="cuda")
    staged = torch.arange(pages * page, dtype=torch.int32, device="cuda")
    q, q_in = torch.zeros_like(c["q"]).cuda(), c["q"].cuda()
    lens, lens_in, sizes = i32([0, 0]), i32(c["lens"]), i32(c["sizes"])
    mask, out = pack_mask(c["seen"]).cuda(), torch.full_like(q, 7.0)
    kept, kept_lens, after = i32([[1, 3, 4, 0, 0, 0, 0, 0]] * 2), i32([3, 2]), i32([0, 0])
    other = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        main = torch.cuda.current_stream()
        k.zero_(), v.zero_(), out.fill_(7.0)                # fills
        slots.copy_(staged)                                 # a copy right before the call
        td.td_kv_append_slots(shape, cache, rows[0], rows[1], slots)
        other.wait_stream(main)
        with torch.cuda.stream(other):
            q.copy_(q_in)
            lens.copy_(lens_in)
        main.wait_stream(other)                             # the call's inputs come from another stream
        td.td_tree_attn(shape, cache, 8, sizes, mask, q, lens, out, ws)
        td.td_tree_commit(shape, [cache], 8, sizes, kept, kept_lens, lens, after, ws)
        lens.zero_()                                        # what the calls read, right behind them
        q.zero_()
    for _ in range(5):
        out.zero_()
        after.zero_()
        g.replay()
    torch.cuda.synchronize()
    check_tree(c, out)
    assert after.tolist() == [900 - 8 + 3, 333 - 5 + 2] and ws.status() == 0
    for b, n in enumerate(c["lens"]):
        ctx = n - c["sizes"][b]
        for i, j in enumerate([1, 3, 4][:3 if b == 0 else 2]):
            at = ctx + i
            assert torch.equal(k[int(c["table"][b, at // page]), :, at % page].cpu(), c["K"][b, :, ctx + j])


@pytest.mark.parametrize("n", [40, 9000])
def test_a_query_row_that_is_not_a_number_says_so(n):
    """In a request that one block does, and in one that is joined from the parts of many."""
    c = tree_case(17, 4, 1, [n], [6], 6, 0, "tree")
    q = c["q"].clone()
    c["q"][0, 2, 1, 7] = float("nan")
    out, ws = run_tree(c)
    row = out[0, 2, 1].clone()
    assert torch.isnan(row).all() and ws.status() == 0
    c["q"] = q
    out[0, 2, 1] = run_tree(c)[0][0, 2, 1]
    check_tree(c, out)


@pytest.mark.parametrize("sparse", [0, 150])
def test_launches_in_plain_stream_order_give_the_same(sparse):
    """With and without programmatic launches, many calls in a row into each other's inputs."""
    c = tree_case(23, 4, 2, [2100, 77, 640], [8, 3, 8], 8, 16, "tree", sparse)
    outs = []
    for pdl in (1, 0):
        td.td_set_tuning("pdl", pdl)
        try:
            out, ws = run_tree(c)
            for _ in range(20):
                run_tree(c, out=out, ws=ws)
            assert ws.status() == 0
        finally:
            td.td_set_tuning("pdl", 1)
        outs.append(out)
    check_tree(c, outs[0])
    assert torch.equal(outs[0], outs[1])
