"""Tree attention where a block takes several units of several tiles each: the
tensor-core work of a unit follows that of the unit before it."""
import pytest
import torch

import sparse_attention_td_gb300 as td
from test_spec_gpu import _built, check_tree, run_tree, tree_case  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("page,k", [(0, 0), (16, 0), (64, 0), (0, 300), (16, 300)])
def test_many_units_of_several_tiles(page, k):
    """320 units of 2 to 5 tiles, 6 to 8 tiles a block: most units begin behind another one."""
    gen = torch.Generator().manual_seed(41 + page + k)
    B, T = 40, 3
    lens = torch.randint(260, 520, (B,), generator=gen).tolist()
    c = tree_case(page + k, 2, 8, lens, [T] * B, T, page, "tree", k, max_len=520)
    out, ws = run_tree(c)
    check_tree(c, out)
    assert ws.status() == 0
    for _ in range(3):
        assert torch.equal(run_tree(c, ws=ws)[0], out)


def test_units_of_one_and_of_several_tiles_in_turn():
    """Every order of one-tile and longer units next to each other in a block."""
    gen = torch.Generator().manual_seed(43)
    B, T = 160, 4
    lens = [T + int(n) for n in torch.randint(0, 400, (B,), generator=gen)]
    lens = [n if b % 3 else T + n % 100 for b, n in enumerate(lens)]
    c = tree_case(44, 4, 4, lens, [T] * B, T, 32, "tree", max_len=416)
    out, ws = run_tree(c)
    check_tree(c, out)
    assert ws.status() == 0
    assert torch.equal(run_tree(c, ws=ws)[0], out)


def test_a_long_launch_is_not_a_stall():
    """The wait limit is one without progress: blocks of about 1700 tiles each, every one of them
    many times longer at work than the limit.  (4M positions on 8 pages that repeat.)"""
    from spec_util import D, E, U
    from test_spec_gpu import i32
    Hkv, T, page, N, P = 8, 2, 128, 1 << 22, 8
    gen = torch.Generator().manual_seed(47)
    blocks = N // page
    table = torch.arange(blocks, dtype=torch.int32).remainder(P).view(1, blocks)
    table[0, -1] = P                                     # the drafted tokens' page
    ctx = (blocks - 1) * page
    k, v = (torch.randn(P + 1, Hkv, page, D, generator=gen).to(torch.bfloat16) for _ in range(2))
    q = torch.randn(1, T, Hkv, D, generator=gen).to(torch.bfloat16)
    shape = td.make_shape(1, Hkv, Hkv, N)
    ws = td.Workspace(shape, 0, tree_size=T)
    x = (shape, td.make_cache(k.cuda(), v.cuda(), table.cuda()), T, None, None, q.cuda(), i32([ctx + T]))
    outs = [torch.full_like(x[5], 7.0) for _ in range(2)]
    td.td_tree_attn(*x, outs[0], ws)
    torch.cuda.synchronize()
    limit = 100
    t0, t1 = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    td.td_set_tuning("wait_limit_us", limit)
    try:
        t0.record()
        td.td_tree_attn(*x, outs[1], ws)
        t1.record()
        torch.cuda.synchronize()
    finally:
        td.td_set_tuning("wait_limit_us", 0)
    assert ws.status() == 0
    assert t0.elapsed_time(t1) * 1e3 > 4 * limit         # else this shows nothing
    assert torch.equal(outs[0], outs[1])
    # Rows of the context count as often as their page comes.  Tolerance as in spec_util, with
    # sums over the tokens of one block of the launch, then over the blocks.
    often = torch.bincount(table[0, :-1].long(), minlength=P).double().repeat_interleave(page)
    n = Hkv * (blocks + 1) // 132 * 128 + 160            # (at least 132 blocks)
    for h in range(Hkv):
        for t in range(T):
            qr = q[0, t, h].double()
            K = torch.cat([k[:P, h].reshape(-1, D), k[P, h, :t + 1]]).double()
            V = torch.cat([v[:P, h].reshape(-1, D), v[P, h, :t + 1]]).double()
            z = (K @ qr) * D ** -0.5
            w = torch.cat([often, torch.ones(t + 1).double()]) * torch.exp(z - z.max())
            w /= w.sum()
            ref, A = w @ V, w @ V.abs()
            ds = D * E * D ** -0.5 * float((K.abs() @ qr.abs()).max())
            dx = 4 * E * float(z.abs().max()) * 1.4427
            tol = U * ref.abs() + (U + 2 * (ds + dx) + 2 * (n + 4) * E) * A * (1 + U)
            assert torch.all((outs[0][0, t, h].cpu().double() - ref).abs() <= tol)
