"""Small-cache calls whose outputs build on the ones before, captured, replayed and queued: every output counts."""
import pytest
import torch

import sparse_attention_td_gb300 as td
from cache_util import D
from test_cache_gpu import Case, _built, i32  # noqa: F401
from test_cache_steps_gpu import calls

pytestmark = pytest.mark.gpu


def below(x, lens):
    """Entries [B][..][n] of positions below each request's length."""
    return torch.cat([x[b, :, :n].flatten() for b, n in enumerate(lens)])


@pytest.mark.parametrize("page,G", [(0, 1), (16, 4), (48, 8)])
def test_weights_of_captured_calls(page, G):
    """All outputs of a replayed call, weights and scores among them."""
    c = Case(101 + G, [300, 140, 1, 2260], G, 2, page)
    run, outs = calls(c, 1, [130, 3, 1, 64])
    for f in run:
        f(None)
    torch.cuda.synchronize()
    want = [o.clone() for o in outs]
    g, st = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(g, stream=st):
        for f in run:
            f(st)
    for _ in range(4):
        for o in outs:
            o.fill_(3.0)
        g.replay()
        for o, r in zip(outs[:3], want):
            assert torch.equal(o, r)
        for o, r in zip(outs[3:], want[3:]):
            assert torch.equal(below(o, c.lens), below(r, c.lens))
    assert c.ws.status() == 0


@pytest.mark.parametrize("pdl", [0, 1])
def test_weights_that_build_up_over_replays(pdl):
    """A captured decode step of two layers adds to its weights at every replay, right behind whatever wrote them."""
    c = Case(103, [500, 17, 2050], 4, 2, 16)
    q = [c.rnd(c.B, 8, D).cuda() for _ in range(2)]
    seq, gen = c.seq, torch.Generator(device="cuda").manual_seed(3)
    out, logits = torch.zeros_like(q[0]), torch.zeros(c.B, 8, c.N, device="cuda")
    w = [torch.zeros(c.B, 2, c.N, device="cuda") for _ in range(2)]
    once = []
    for x in q:                                          # what one call adds
        s = torch.zeros(c.B, 2, c.N, device="cuda")
        td.td_weights_attn(c.shape, c.cache, c.N, x, seq, s, logits, out, c.ws)
        once.append(s)
    torch.cuda.synchronize()
    td.td_set_tuning("pdl", pdl)
    try:
        g, st = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        with torch.cuda.graph(g, stream=st):
            for _ in range(3):
                for x, s in zip(q, w):
                    td.td_weights_attn(c.shape, c.cache, 1, x, seq, s, logits, out, c.ws, st)
        for _ in range(3):
            old = [torch.rand(s.shape, generator=gen, device="cuda") for s in w]
            want = []
            for s, o, a in zip(w, old, once):
                t = o.clone()
                for _ in range(3):
                    for b, n in enumerate(c.lens):
                        t[b, :, n - 1] = 0.0
                    t = t + a
                want.append(t)
            torch.cuda.synchronize()
            for s, o in zip(w, old):
                s.copy_(o)
            g.replay()
            for s, t in zip(w, want):
                # (three times G + 1 sums on either side, each off by 2^-24 of the largest result at most)
                s, t = below(s, c.lens), below(t, c.lens)
                assert (s - t).abs().max().item() <= 3 * (4 + 1) * 2 * 2.0 ** -24 * t.max().item()
    finally:
        td.td_set_tuning("pdl", 1)
    assert c.ws.status() == 0


def test_two_streams_and_their_weights():
    """Calls of two requests' sets at once, each with its workspace: weights and scores as alone."""
    cases = [Case(105, [900, 500], 4, 2, 16), Case(106, [700, 650, 10], 8, 1, 0)]
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
    for (_, outs), ref, c in zip(jobs, want, cases):
        assert all(torch.equal(o, r) for o, r in zip(outs[:3], ref)) and c.ws.status() == 0
        assert all(torch.equal(below(o, c.lens), below(r, c.lens)) for o, r in zip(outs[3:], ref[3:]))


def test_a_captured_step_with_eviction():
    """Append, weights and eviction in place, captured once and replayed for every step, against the same calls one
    by one: whole caches, weights, kept positions and lengths."""
    B, Hkv, G, N, budget = 3, 2, 4, 1300, 1200

    def setup():
        c = Case(107, [budget] * B, G, Hkv, 16, N=N)
        c.table = torch.arange(B * c.table.shape[1], dtype=torch.int32).view(B, -1)
        c.dev_table.copy_(c.table)
        for x in c.parts:
            x.nan_to_num_(0.5, 0.5, 0.5)
        gen = torch.Generator(device="cuda").manual_seed(9)
        s = dict(c=c, q=torch.zeros(B, G * Hkv, D, dtype=torch.bfloat16, device="cuda"),
                 new=torch.zeros(B, 2, Hkv, D, dtype=torch.bfloat16, device="cuda"),
                 seq=i32([budget + 1] * B), seq_out=i32([0] * B), logits=torch.zeros(B, G * Hkv, N, device="cuda"),
                 w=torch.rand(B, Hkv, N, generator=gen, device="cuda"),
                 kept=torch.zeros(B, Hkv, budget, dtype=torch.int32, device="cuda"),
                 slots=torch.tensor([int(c.table[b, budget // 16]) * 16 + budget % 16 for b in range(B)], dtype=torch.int32).cuda())
        s["out"] = torch.zeros_like(s["q"])
        return s

    def step(s, st=None):
        c = s["c"]
        td.td_kv_append_slots(c.shape, c.cache, s["new"][:, 0], s["new"][:, 1], s["slots"], st)
        td.td_weights_attn(c.shape, c.cache, 1, s["q"], s["seq"], s["w"], s["logits"], s["out"], c.ws, st)
        td.td_evict(c.shape, c.cache, c.cache, budget, 4, 100, s["w"], s["w"], s["seq"], s["seq_out"], s["kept"], c.ws, st)
    one, two = setup(), setup()
    g, st = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(g, stream=st):
        step(two, st)
    gen = torch.Generator(device="cuda").manual_seed(11)
    for i in range(6):
        q = torch.randn(one["q"].shape, generator=gen, device="cuda").to(torch.bfloat16)
        new = torch.randn(one["new"].shape, generator=gen, device="cuda").to(torch.bfloat16)
        for s in (one, two):
            s["q"].copy_(q)
            s["new"].copy_(new)
        step(one)
        torch.cuda.synchronize()
        g.replay()
        for name in ("out", "kept", "seq_out", "w"):
            assert torch.equal(one[name], two[name]), (i, name)
        assert all(torch.equal(x, y) for x, y in zip(one["c"].parts, two["c"].parts)), i
        assert one["kept"][:, :, -1].eq(budget).all() and one["seq_out"].tolist() == [budget] * B
    assert one["c"].ws.status() == 0 and two["c"].ws.status() == 0
