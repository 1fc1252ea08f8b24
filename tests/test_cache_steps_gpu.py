"""Operators on small caches together, as a serving loop uses them: steps whose calls read what the
ones before wrote, captured graphs, streams, shared workspaces, and the failure report."""
import pytest
import torch

import sparse_attention_td_gb300 as td
from cache_util import D, U, attend, evict, quantise, values, visible
from test_cache_gpu import Case, _built, call, i32, near, run_new  # noqa: F401

pytestmark = pytest.mark.gpu


# --------------------------------------------------- serving over a 4-bit cache
class Server:
    """Requests on 4-bit pages: each step has new tokens of some requests."""

    def __init__(self, seed, B, Hkv, G, page, N):
        self.gen = torch.Generator().manual_seed(seed)
        self.B, self.Hkv, self.G, self.page, self.N = B, Hkv, G, page, N
        blocks = -(-N // page)
        P = B * blocks
        self.shape = td.make_shape(B, G * Hkv, Hkv, N)
        self.parts = [torch.full((P, Hkv, page, w), 0xff, dtype=torch.uint8).cuda() for w in (64, 64, 16)]
        self.table = torch.full((B, blocks), -1, dtype=torch.int32).cuda()
        self.cache = td.make_q4_cache(*self.parts, self.table)
        self.held, self.count = i32([0] * B), i32([P])
        self.free = torch.randperm(P, generator=self.gen).to(torch.int32).cuda()
        self.ws = td.Workspace(self.shape, 0, cache_calls=True)
        self.lens = [0] * B
        self.rows = [[] for _ in range(B)]            # per request: (K, V) [Hkv][D] of each token, in 64 bits

    def step(self, new, window, sinks):
        """One step with new[b] new tokens; returns the outputs, which are checked."""
        rnd = lambda *s: torch.randn(*s, generator=self.gen).to(torch.bfloat16)
        total = sum(new)
        self.lens = [n + t for n, t in zip(self.lens, new)]
        kv, q = rnd(total, 2, self.Hkv, D), 2 * rnd(total, self.G * self.Hkv, D)
        seq = i32(self.lens)
        cu, slots = i32([0] * (self.B + 1)), i32([0] * total)
        out = torch.full_like(q, 7.0).cuda()
        kvd, qd = kv.cuda(), q.cuda()
        td.td_block_tables(seq, i32(new), self.page, self.table, self.held, self.held, self.free, self.count,
                           self.count, cu, slots, ws=self.ws)
        td.td_q4_append(self.shape, self.cache, kvd[:, 0], kvd[:, 1], slots)
        td.td_q4_attn(self.shape, self.cache, window, sinks, cu, qd, seq, out, ws=self.ws)
        at = 0
        for b, t in enumerate(new):
            for i in range(t):
                self.rows[b].append([values(*quantise(kv[at + i, j])) for j in range(2)])
            at += t
        at = 0
        for b, t in enumerate(new):
            n = self.lens[b]
            if not t:
                continue
            K = torch.stack([r[0] for r in self.rows[b]])
            V = torch.stack([r[1] for r in self.rows[b]])
            sees = torch.zeros(t, n, dtype=torch.bool)
            for i in range(t):
                sees[i, visible(n, n - t + i, window, sinks)] = True
            for h in range(self.G * self.Hkv):
                ref, tol, _, _ = attend(q[at:at + t, h], K[:, h // self.G], V[:, h // self.G], sees, 2.0 ** -11, True)
                near(out[at:at + t, h], ref, tol)
            at += t
        assert self.ws.status() == 0
        if all(t == 1 for t in new):                  # a decode step: the single-token form agrees
            one = torch.zeros_like(out)
            td.td_q4_attn(self.shape, self.cache, window, sinks, None, qd, seq, one, ws=self.ws)
            assert (one.float() - out.float()).abs().max().item() <= 2.0 ** -7 * out.float().abs().max().item()


@pytest.mark.parametrize("page,window,sinks", [(16, 0, 0), (8, 40, 3), (48, 100, 1)])
def test_serving_over_a_4_bit_cache(page, window, sinks):
    s = Server(page, 4, 2, 4, page, 400)
    for new in ([130, 1, 33, 0], [1, 1, 1, 200], [1, 1, 1, 1], [1, 64, 0, 1], [1, 1, 1, 1]):
        s.step(new, window, sinks)


# --------------------------------------------------- decoding with eviction
@pytest.mark.parametrize("page", [0, 16])
def test_decoding_with_eviction(page):
    """Every step appends a token, attends with weights and evicts back to the budget."""
    B, Hkv, G, N, budget, sinks, recent = 3, 2, 2, 80, 64, 2, 16
    c = Case(21 + page, [70, 20, 64], G, Hkv, page, N=N)
    if page:                                          # all blocks of the table are used here
        c.table = torch.arange(B * c.table.shape[1], dtype=torch.int32).view(B, -1).flip(1).contiguous()
        c.dev_table.copy_(c.table)
    lens = [64, 20, 63]
    at = lambda b, p: (b, p) if not page else (int(c.table[b, p // page]), p % page)
    for x, fresh in zip(c.parts, (c.rnd(B, N, Hkv, D), c.rnd(B, N, Hkv, D))):
        for b in range(B):
            for p in range(N):
                i, r = at(b, p)
                x[i, :, r] = fresh[b, p].cuda()
    w = torch.rand(B, Hkv, N, generator=c.gen).cuda()
    logits = torch.zeros(B, G * Hkv, N).cuda()
    kept = torch.zeros(B, Hkv, budget, dtype=torch.int32).cuda()
    seq_out = i32(lens)
    for step in range(9):
        lens = [n + 1 for n in lens]
        seq = i32(lens)
        new = c.rnd(B, 2, Hkv, D).cuda()
        slots = []
        for b, n in enumerate(lens):
            i, r = at(b, n - 1)
            slots.append(i * (page or N) + r)
        td.td_kv_append_slots(c.shape, c.cache, new[:, 0], new[:, 1], i32(slots))
        q = 2 * c.rnd(B, G * Hkv, D)
        out = torch.zeros_like(q).cuda()
        w0 = w.clone()
        td.td_weights_attn(c.shape, c.cache, 1, q.cuda(), seq, w, logits, out, ws=c.ws)
        rows = lambda x, b, g: torch.stack([x[at(b, p)[0], g, at(b, p)[1]] for p in range(lens[b])]).cpu()
        before = [[(rows(c.parts[0], b, g), rows(c.parts[1], b, g)) for g in range(Hkv)] for b in range(B)]
        for b, n in enumerate(lens):
            for g in range(Hkv):
                K, V = before[b][g]
                total = w0[b, g, :n].cpu().double()
                total[n - 1] = 0
                bound = torch.zeros(n, dtype=torch.float64)
                for h in range(g * G, (g + 1) * G):
                    ref, tol, a, rel = attend(q[b:b + 1, h], K.double(), V.double(), torch.ones(1, n, dtype=torch.bool), U * U)
                    near(out[b:b + 1, h], ref, tol)
                    total += a[0]
                    bound += a[0] * rel[0]
                near(w[b, g, :n], total, bound + 3 * 2.0 ** -23 * total)
        w1 = w.cpu()
        td.td_evict(c.shape, c.cache, c.cache, budget, sinks, recent, w, w, seq, seq_out, kept, ws=c.ws)
        assert c.ws.status() == 0
        for b, n in enumerate(lens):
            for g in range(Hkv):
                keep = evict(w1[b, g].tolist(), n, budget, sinks, recent)
                assert kept[b, g].tolist() == keep + [-1] * (budget - len(keep))
                assert torch.equal(w[b, g, :len(keep)].cpu(), w1[b, g, keep])
                for x, old in zip(c.parts, before[b][g]):
                    now = torch.stack([x[at(b, p)[0], g, at(b, p)[1]] for p in range(len(keep))]).cpu()
                    assert torch.equal(now, old[keep])
        lens = seq_out.tolist()
        assert lens == [min(n, budget) for n in seq.tolist()]


# --------------------------------------------------- graphs, streams, workspaces
def calls(c, seed, new):
    """Closures of one call of each kind on case c, and their outputs."""
    gen = torch.Generator().manual_seed(seed)
    total = sum(new)
    q = torch.randn(total, c.G * c.Hkv, D, generator=gen).to(torch.bfloat16).cuda()
    q1 = q[:c.B].contiguous()
    cu = i32([0] + torch.tensor(new).cumsum(0).tolist())
    outs = [torch.zeros_like(q), torch.zeros_like(q1), torch.zeros_like(q1)]
    run = [lambda s: call(c)(c.shape, c.cache, 70, 2, cu, q, c.seq, outs[0], c.ws, s),
           lambda s: call(c)(c.shape, c.cache, 0, 0, None, q1, c.seq, outs[1], c.ws, s)]
    if c.q4:
        k = min(c.lens + [40])                        # positions that every request has
        idx = torch.arange(k, dtype=torch.int32).expand(c.B, c.Hkv, k).contiguous().cuda()
        run.append(lambda s: td.td_q4_sparse_attn(c.shape, c.cache, q1, c.seq, idx, k, outs[2], c.ws, s))
    else:
        w = torch.zeros(c.B, c.Hkv, c.N).cuda()
        logits = torch.zeros(c.B, c.G * c.Hkv, c.N).cuda()
        outs += [w, logits]
        run.append(lambda s: td.td_weights_attn(c.shape, c.cache, c.N, q1, c.seq, w, logits, outs[2], c.ws, s))
    return run, outs


@pytest.mark.parametrize("q4", [False, True])
def test_captured_calls_that_share_a_workspace(q4):
    """Two graphs of calls of every kind on one workspace, replayed in turn, give what eager calls give."""
    cases = [Case(31, [300, 140, 260], 4, 2, 16, q4), Case(32, [600], 2, 1, 0, q4)]
    ws = td.Workspace(cases[0].shape, 0, cache_calls=True)
    want, graphs = [], []
    st = torch.cuda.Stream()
    for k, c in enumerate(cases):
        c.ws = ws
        run, outs = calls(c, k, [130, 3, 64] if k == 0 else [200])
        for f in run:
            f(None)
        torch.cuda.synchronize()
        want.append([o.clone() for o in outs])
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            for f in run:
                f(st)
        graphs.append((g, outs, run))                 # (run holds the inputs)
    for _ in range(4):
        for (g, outs, _), ref in zip(graphs, want):
            for o in outs:
                o.fill_(3.0)
            g.replay()
            for o, r in zip(outs[:3], ref):
                assert torch.equal(o, r)
    assert ws.status() == 0


@pytest.mark.parametrize("q4", [False, True])
def test_streams_with_their_own_workspaces(q4):
    cases = [Case(41, [900, 500], 4, 2, 16, q4), Case(42, [700, 650, 10], 8, 1, 0, q4)]
    jobs = [calls(c, k, [120, 200] if k == 0 else [300, 1, 10]) for k, c in enumerate(cases)]
    want = []
    for run, outs in jobs:
        for f in run:
            f(None)
        torch.cuda.synchronize()
        want.append([o.clone() for o in outs])
        for o in outs:
            o.zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for it in range(6):
        for i in ((0, 1) if it % 2 else (1, 0)):
            for f in jobs[i][0]:
                f(streams[i])
    torch.cuda.synchronize()
    for (run, outs), ref, c in zip(jobs, want, cases):
        assert all(torch.equal(o, r) for o, r in zip(outs[:3], ref)) and c.ws.status() == 0


@pytest.mark.parametrize("pdl", [0, 1])
def test_calls_queued_behind_one_another(pdl):
    """Each call's query is the output of the one before: programmatic launches change nothing."""
    c = Case(51, [500, 333], 4, 2, 16)
    q0 = c.rnd(2, 8, D).cuda()
    cu = i32([0, 1, 2])
    outs = []
    td.td_set_tuning("pdl", pdl)
    try:
        for wait in (False, True):
            q = q0.clone()
            for i in range(12):
                out = torch.zeros_like(q)
                td.td_window_attn(c.shape, c.cache, 100 + 40 * i, 3, cu if i % 3 == 1 else None, q, c.seq, out, c.ws)
                if wait:
                    torch.cuda.synchronize()
                q = out
            outs.append(q)
    finally:
        td.td_set_tuning("pdl", 1)
    assert torch.equal(*outs)


def test_one_workspace_for_every_kind_of_call():
    """Selection, tree calls and the calls on small caches in turn on one workspace with a part for each."""
    c = Case(61, [600, 444], 4, 2, 0)
    K, V = c.parts[0].nan_to_num(0.0, 0.0, 0.0), c.parts[1].nan_to_num(0.0, 0.0, 0.0)
    cache = td.make_cache(K, V)
    k, T = 64, 5
    ws = td.Workspace(c.shape, k, tree_size=T, cache_calls=True)
    q = c.rnd(2, 8, D).cuda()
    qt = c.rnd(2, T, 8, D).cuda()

    def run(ws):
        idx = torch.full((2, 2, k), -1, dtype=torch.int32).cuda()
        outs = [torch.zeros_like(q), torch.zeros_like(qt), torch.zeros_like(q), torch.zeros_like(q)]
        td.td_full_attn_select(c.shape, q, K, V, c.seq, k, idx, outs[0], ws=ws)
        td.td_tree_attn(c.shape, cache, T, None, None, qt, c.seq, outs[1], ws=ws)
        td.td_window_attn(c.shape, cache, 200, 2, None, q, c.seq, outs[2], ws=ws)
        td.td_window_attn(c.shape, cache, 200, 2, i32([0, 1, 2]), q, c.seq, outs[3], ws=ws)
        return [idx] + outs
    first = run(ws)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(run(ws), first))
    assert ws.status() == 0
    td.td_window_attn(c.shape, cache, 200, 2, None, q, c.seq, first[3], ws=td.Workspace(c.shape, 0, cache_calls=True))
    with pytest.raises(ValueError, match="cache_calls"):
        td.td_window_attn(c.shape, cache, 1, 0, None, q, c.seq, torch.zeros_like(q), ws=td.Workspace(c.shape, k, tree_size=T))
    with pytest.raises(ValueError, match="cache_calls"):
        big = td.make_shape(500, 8, 2, 600)
        td.td_weights_attn(big, td.make_cache(K, V, c.seq.view(2, 1)), 1, q, c.seq, q, q, q, ws=ws)


def test_arguments_are_checked():
    c, c4 = Case(71, [60, 50], 4, 2, 16), Case(72, [60, 50], 4, 2, 16, True)
    q, out = c.rnd(2, 8, D).cuda(), torch.zeros(2, 8, D, dtype=torch.bfloat16).cuda()
    with pytest.raises(ValueError):
        td.td_window_attn(c.shape, c4.cache, 1, 0, None, q, c.seq, out, c.ws)
    with pytest.raises(ValueError):
        td.td_q4_attn(c.shape, c.cache, 1, 0, None, q, c.seq, out, c.ws)
    with pytest.raises(ValueError):
        td.td_window_attn(c.shape, c.cache, 1, 0, None, q.view(2, 4, 256), c.seq, out, c.ws)
    with pytest.raises(ValueError):
        td.td_window_attn(c.shape, c.cache, 1, 0, None, q.float(), c.seq, out, c.ws)
    with pytest.raises(ValueError):
        td.td_window_attn(c.shape, c.cache, 1, 0, None, q.cpu(), c.seq, out, c.ws)
    with pytest.raises(ValueError):
        td.td_window_attn(c.shape, c.cache, 1, 0, i32([0, 1]), q, c.seq, out, c.ws)      # cu_new too short
    with pytest.raises(ValueError):
        td.td_window_attn(c.shape, c.cache, 1, 0, None, q, c.seq, out[:1], c.ws)
    with pytest.raises(td.TdError):
        td.td_window_attn(c.shape, c.cache, -1, 0, None, q, c.seq, out, c.ws)
    with pytest.raises(td.TdError):
        td.td_window_attn(c.shape, c.cache, 1, 0, None, q[:1], c.seq, out, c.ws)         # not one per request
    with pytest.raises(ValueError):
        td.make_q4_cache(c4.parts[0], c4.parts[1], c4.parts[2][:, :, :, :8].contiguous())
    with pytest.raises(ValueError):
        td.make_q4_cache(c4.parts[0], c4.parts[1][:1], c4.parts[2])
    assert torch.all(out == 0.0)


# --------------------------------------------------- the failure report
@pytest.mark.parametrize("q4", [False, True])
@pytest.mark.parametrize("bad", [[0, 400, 0, 400], [400, 30, 200, 20], [-5, 10, 1 << 30, 7], [400, 400, 400, 0]])
def test_wrong_borders_then_the_next_call_is_right(bad, q4):
    """A cu_new that does not ascend: its rows are anyone's, but nothing else is touched."""
    c = Case(71, [500, 333, 290], 4, 2, 16, q4)
    q = c.rnd(400, 8, D).cuda()
    run = td.td_q4_attn if q4 else td.td_window_attn
    out = torch.zeros(402, 8, D, dtype=torch.bfloat16, device="cuda")
    run(c.shape, c.cache, 200, 3, i32(bad), q, c.seq, out[1:401], c.ws)
    torch.cuda.synchronize()
    assert not out[0].any() and not out[401].any() and not c.ws.status() & td.FLAG_WAIT_TIMEOUT
    good = i32([0, 100, 400, 400])
    got, want = torch.zeros_like(q), torch.zeros_like(q)
    run(c.shape, c.cache, 200, 3, good, q, c.seq, got, c.ws)
    run(c.shape, c.cache, 200, 3, good, q, c.seq, want, td.Workspace(c.shape, 0, cache_calls=True))
    assert torch.equal(got, want) and got[100:].any()


@pytest.mark.parametrize("q4", [False, True])
@pytest.mark.parametrize("new", [[100, 300], [1, 1], [700, 3]])
def test_wait_runs_out_then_the_next_call_is_right(new, q4):
    """The softmax waits for what nothing arrives on: the CTAs give up, report it and leave, and the
    next call on the workspace is right."""
    c = Case(sum(new), [900, 400], 4, 2, 16, q4)
    out = run_new(c, new, 0, 0)
    q = torch.zeros_like(out)
    td.td_set_tuning("wait_limit_us", 20)
    td.td_set_tuning("wait_test", 1)
    try:
        cu = i32([0, new[0], sum(new)])
        call(c)(c.shape, c.cache, 0, 0, cu, q, c.seq, torch.zeros_like(q), c.ws)
        torch.cuda.synchronize()
    finally:
        td.td_set_tuning("wait_test", 0)
        td.td_set_tuning("wait_limit_us", 0)
    assert c.ws.status() == td.FLAG_WAIT_TIMEOUT
    run_new(c, new, 0, 0)
