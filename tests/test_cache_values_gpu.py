"""Values that are not finite in small caches: what they cost, and whom they reach."""
import pytest
import torch

import sparse_attention_td_gb300 as td
from cache_util import D, U, attend, visible
from test_cache_gpu import Case, _built, call, i32, near  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("q4", [False, True])
@pytest.mark.parametrize("dims", [16, 128])
def test_rows_done_again_outlast_no_wait(dims, q4):
    """Prompts between others whose every row sees a value of which some or all dims are NaN: those rows are
    computed once more, one by one, and take (in some dims) far longer than a wait without progress may."""
    n, Hkv, G = 600, 8, 4
    c = Case(81, [n] * 8, G, Hkv, 0, q4)
    for b in (0, 2, 5, 6):
        if q4:
            c.parts[2][b, :, 3, 8:8 + dims // 16] = 0x7f
        else:
            c.parts[1][b, :, 3, :dims] = float("nan")
    q = 2 * c.rnd(8 * n, Hkv * G, D)
    out = torch.zeros_like(q).cuda()
    cu = i32([n * b for b in range(9)])
    td.td_set_tuning("wait_limit_us", 500)
    try:
        call(c)(c.shape, c.cache, 0, 0, cu, q.cuda(), c.seq, out, c.ws)
        torch.cuda.synchronize()
    finally:
        td.td_set_tuning("wait_limit_us", 0)
    assert c.ws.status() == 0
    sees = torch.ones(n, n, dtype=torch.bool).tril()
    for b in range(8):
        rows = slice(n * b, n * b + n)
        if b in (0, 2, 5, 6):
            assert out[rows][3:, :, :dims].isnan().all() and out[rows][:3].isfinite().all()
            assert out[rows][3:, :, dims:].isfinite().all()
            continue
        for h in (0, 13, 31):
            ref, tol, _, _ = attend(q[rows, h], c.K[b, h // G], c.V[b, h // G], sees, 2.0 ** -11 if q4 else U, q4)
            near(out[rows, h], ref, tol)


@pytest.mark.parametrize("q4", [False, True])
@pytest.mark.parametrize("lens,new,window,sinks", [([203, 131, 90, 77] * 20, [50, 64, 1, 13] * 20, 37, 5),
                                                   ([203, 131, 90, 77] * 20, [50, 64, 1, 13] * 20, 0, 0),
                                                   ([3001, 2050], [30, 9], 0, 0), ([3001, 2050], [30, 9], 1003, 2)])
def test_rows_done_again_are_right(lens, new, window, sinks, q4):
    """The last token's value is a NaN that no row but its own sees: the rows beside it are computed one by one, in
    whole units and in ones that several CTAs share, over pages of which one is none."""
    c = Case(83, lens, 2, 1, 16, q4)
    for b, n in enumerate(lens):
        at = (int(c.table[b, (n - 1) // 16]), 0, (n - 1) % 16)
        if q4:
            c.parts[2][at][8:] = 0x7f
        else:
            c.parts[1][at] = float("nan")
    gone = range(16, 32)
    c.dev_table[:, 1] = -1
    q = 2 * c.rnd(sum(new), 2, D)
    out = torch.zeros_like(q).cuda()
    cu = [0]
    for t in new:
        cu.append(cu[-1] + t)
    call(c)(c.shape, c.cache, window, sinks, i32(cu), q.cuda(), c.seq, out, c.ws)
    assert c.ws.status() == (0 if window and all(n - t - window >= 32 for n, t in zip(lens, new)) else td.FLAG_PAGE_OUT_OF_RANGE)
    last = torch.zeros(len(q), dtype=torch.bool)
    last[[e - 1 for e in cu[1:]]] = True
    assert out[last].isnan().all()
    ref, tol = c.attend(q, [(b, list(range(n - t, n))) for b, (n, t) in enumerate(zip(lens, new))],
                        lambda b, g, p: [j for j in visible(lens[b], p, window, sinks) if j not in gone],
                        2.0 ** -11 if q4 else U)
    near(out[~last], ref[~last], tol[~last])


@pytest.mark.parametrize("q4", [False, True])
def test_windows_and_sinks_of_the_largest_size(q4):
    """max_seq_len = 2^30 over a table of one page, a window and first tokens that add up to 2^31 - 1."""
    page, blocks, n = 1 << 16, 1 << 14, 300
    shape = td.make_shape(1, 4, 1, page * blocks)
    c = Case(84, [n], 4, 1, 0, q4)
    parts = []
    for x in c.parts:
        big = torch.zeros(1, 1, page, x.shape[3], dtype=x.dtype, device="cuda")
        big[:, :, :n] = x
        parts.append(big)
    table = torch.zeros(1, blocks, dtype=torch.int32, device="cuda")
    cache = td.make_q4_cache(*parts, table) if q4 else td.make_cache(*parts, table)
    ws = td.Workspace(td.make_shape(1, 4, 1, n), 0, cache_calls=True)
    for T, cu in ((1, None), (40, i32([0, 40]))):
        q = 2 * c.rnd(T, 4, D)
        out = torch.zeros_like(q).cuda()
        call(c)(shape, cache, (1 << 30) - 1, 1 << 30, cu, q.cuda(), c.seq, out, ws)
        ref, tol = c.attend(q, [(0, list(range(n - T, n)))], lambda b, g, p: list(range(p + 1)), 2.0 ** -11 if q4 else U)
        near(out, ref, tol)
    assert ws.status() == 0
