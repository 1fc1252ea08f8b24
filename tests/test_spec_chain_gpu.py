"""Speculative-decoding calls queued behind one another without a wait of the host, each reading
what the one before it wrote, and keys that are not numbers."""
import pytest
import torch

import sparse_attention_td_gb300 as td
from spec_util import D, pack_mask
from test_spec_gpu import _built, check_tree, i32, run_tree, tree_case  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("ctx", [0, 70, 256, 9088])
def test_a_key_that_is_not_a_number_reaches_the_rows_that_see_it(ctx):
    """... and only those; in one block, and joined from parts."""
    T = 5
    c = tree_case(ctx + 1, 2, 1, [ctx + T], [T], T, 0, "tree")
    c["seen"][0, :, 3] = False
    c["seen"][0, 4, 3] = True                     # the last row alone sees token 3
    cc = dict(c, K=c["K"].clone())
    cc["K"][0, 0, ctx + 3, 11] = float("nan")
    cc["kc"] = cc["K"]
    got, ws = run_tree(cc)
    clean, _ = run_tree(c)
    check_tree(c, clean)
    assert torch.isnan(got[0, 4]).all()
    assert torch.equal(got[0, :4], clean[0, :4])
    assert ws.status() == 0


@pytest.mark.parametrize("sparse", [0, 150])
def test_a_chain_of_calls_each_reading_what_the_one_before_wrote(sparse):
    """Twelve steps queued at once: block tables, the append of rows that the last attention gave,
    attention whose output is the next step's query, the commit whose lengths the next step takes.
    With and without programmatic launches, and with the host waiting between any two calls."""
    B, G, Hkv, T, page, N, steps = 3, 4, 2, 6, 16, 900, 12
    gen = torch.Generator().manual_seed(51 + sparse)
    blocks = -(-N // page)
    pages = B * blocks
    shape = td.make_shape(B, G * Hkv, Hkv, N)
    start = [700, 77, 340]
    perm = torch.randperm(pages, generator=gen).to(torch.int32)
    k0, v0 = (torch.randn(pages, Hkv, page, D, generator=gen).to(torch.bfloat16).cuda() for _ in range(2))
    q0 = (2 * torch.randn(B, T, G * Hkv, D, generator=gen)).to(torch.bfloat16).cuda()
    held0 = [-(-n // page) for n in start]
    table0 = torch.full((B, blocks), -1, dtype=torch.int32)
    used = 0
    for b in range(B):
        table0[b, :held0[b]] = perm[used:used + held0[b]]
        used += held0[b]
    free0 = torch.zeros(pages, dtype=torch.int32)
    free0[:pages - used] = perm[used:]
    seen = torch.ones(T, T, dtype=torch.bool).tril().expand(B, T, T).clone()
    seen[:, 4, 2] = False
    mask = pack_mask(seen).cuda()
    acc, kept, grow = i32([[0, 2, 3, 5, 0, 0]] * B), i32([4, 1, 2]), i32([T] * B)
    idx = None
    if sparse:
        idx = torch.stack([torch.stack([torch.randperm(min(n, 500), generator=gen)[:70] for _ in range(Hkv)])
                           for n in start]).to(torch.int32).cuda()

    def run(pdl, wait):
        k, v, table, held = k0.clone(), v0.clone(), table0.cuda(), i32(held0)
        free, count, cu = free0.cuda(), i32([pages - used]), i32([0] * (B + 1))
        slots = i32([-9] * (B * T))
        seq, lens = i32(start), i32([0] * B)
        ws = td.Workspace(shape, 0, tree_size=T)
        cache = td.make_cache(k, v, table)
        a, o = q0.clone(), torch.full_like(q0, 7.0)
        td.td_set_tuning("pdl", pdl)
        sync = torch.cuda.synchronize if wait else lambda: None
        torch.cuda.synchronize()
        try:
            for _ in range(steps):
                torch.add(seq, grow, out=lens)
                sync()
                td.td_block_tables(lens, grow, page, table, held, held, free, count, count, cu, slots, ws)
                sync()
                rows = a.view(B * T, G * Hkv, D)           # the last output's heads as new rows
                td.td_kv_append_slots(shape, cache, rows[:, :Hkv], rows[:, Hkv:2 * Hkv], slots)
                sync()
                if idx is None:
                    td.td_tree_attn(shape, cache, T, None, mask, a, lens, o, ws)
                else:
                    td.td_tree_sparse_attn(shape, cache, T, None, mask, a, lens, idx, 70, o, ws)
                sync()
                td.td_tree_commit(shape, [cache], T, None, acc, kept, lens, seq, ws)
                sync()
                a, o = o, a
            torch.cuda.synchronize()
        finally:
            td.td_set_tuning("pdl", 1)
        assert ws.status() == 0
        return a, o, k, v, table, held, count, seq, slots

    waited = run(0, True)
    assert waited[7].tolist() == [n + steps * m for n, m in zip(start, [4, 1, 2])]
    for pdl in (1, 0):
        for _ in range(3):
            for x, y in zip(run(pdl, False), waited):
                assert torch.equal(x, y)
