"""Operators on small caches on the GPU against plain references."""
import pytest
import torch

import sparse_attention_td_gb300 as td
from cache_util import D, E, U, attend, evict, paged, quantise, values, visible

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)


def i32(x):
    return torch.as_tensor(x, dtype=torch.int32).cuda()


class Case:
    """A cache of ragged requests; every row that holds no token of a request is not finite."""

    def __init__(self, seed, lens, G=4, Hkv=2, page=0, q4=False, spare=3, N=None):
        gen = self.gen = torch.Generator().manual_seed(seed)
        self.lens, self.G, self.Hkv, self.page, self.q4 = lens, G, Hkv, page, q4
        B = self.B = len(lens)
        N = self.N = N or max(max(lens), 1)
        self.rnd = lambda *s: torch.randn(*s, generator=gen).to(torch.bfloat16)
        K, V = self.rnd(B, Hkv, N, D), self.rnd(B, Hkv, N, D)
        self.table = None
        if page:
            blocks = -(-N // page)
            self.pages = B * blocks + spare
            self.table = torch.randperm(self.pages, generator=gen)[:B * blocks].view(B, blocks).to(torch.int32)
        put = lambda x, fill: paged(x, page, self.table, self.pages, fill) if page else x
        if q4:
            (kc, ks), (vc, vs) = quantise(K), quantise(V)
            self.K, self.V = values(kc, ks), values(vc, vs)
            sc = torch.cat([ks, vs], -1)
            for b, n in enumerate(lens):
                sc[b, :, n:] = 0x7f
            self.parts = [put(kc, 255).cuda(), put(vc, 255).cuda(), put(sc, 0x7f).cuda()]
            make = td.make_q4_cache
        else:
            for b, n in enumerate(lens):
                K[b, :, n:] = float("nan")
                V[b, :, n:] = float("inf")
            self.K, self.V = K, V
            self.parts = [put(K, float("nan")).cuda(), put(V, float("inf")).cuda()]
            make = td.make_cache
        if page:
            for b, n in enumerate(lens):       # entries beyond the length are not read
                self.table[b, -(-n // page):] = 1 << 30
        self.shape = td.make_shape(B, G * Hkv, Hkv, N)
        self.dev_table = None if self.table is None else self.table.cuda()
        self.cache = make(*self.parts, self.dev_table)
        self.seq = i32(lens)
        self.ws = td.Workspace(self.shape, 0, cache_calls=True)

    def attend(self, q, positions, sees_of, pu):
        """Reference of rows q [T][Hq][D] of request b at `positions`, (b, positions) pairs in order."""
        out, tol = torch.zeros(q.shape, dtype=torch.float64), torch.zeros(q.shape, dtype=torch.float64)
        at = 0
        for b, ps in positions:
            for g in range(self.Hkv):
                n = self.lens[b]
                sees = torch.zeros(len(ps), n, dtype=torch.bool)
                for t, p in enumerate(ps):
                    sees[t, sees_of(b, g, p)] = True
                rows = slice(at, at + len(ps))
                for h in range(g * self.G, (g + 1) * self.G):
                    o, e, _, _ = attend(q[rows, h], self.K[b, g, :n].double(), self.V[b, g, :n].double(), sees, pu,
                                        self.q4)
                    out[rows, h], tol[rows, h] = o, e
            at += len(ps)
        return out, tol


def near(got, ref, tol):
    err = (got.cpu().double() - ref).abs()
    worst = (err - tol).max().item() if err.numel() else 0.0
    assert worst <= 0 and not err.isnan().any(), f"error {err.max().item():.3e}, {worst:.3e} over its tolerance"


def call(c):
    return td.td_q4_attn if c.q4 else td.td_window_attn


def run_tokens(c, window, sinks, pu=None):
    q = 2 * c.rnd(c.B, c.G * c.Hkv, D)
    out = torch.full_like(q, 7.0).cuda()
    call(c)(c.shape, c.cache, window, sinks, None, q.cuda(), c.seq, out, c.ws)
    pu = pu or (2.0 ** -11 if c.q4 else U * U)
    ref, tol = c.attend(q, [(b, [n - 1]) for b, n in enumerate(c.lens)],
                        lambda b, g, p: visible(c.lens[b], p, window, sinks), pu)
    near(out, ref, tol)
    assert c.ws.status() == 0
    return out


def run_new(c, new, window, sinks, tail=0, lead=0):
    """new[b] new tokens per request in a packed batch (rows before and behind them belong to nobody)."""
    total = sum(new)
    q = 2 * c.rnd(lead + total + tail, c.G * c.Hkv, D)
    cu = [lead]
    for t in new:
        cu.append(cu[-1] + t)
    out = torch.full_like(q, 7.0).cuda()
    call(c)(c.shape, c.cache, window, sinks, i32(cu), q.cuda(), c.seq, out, c.ws)
    ref, tol = c.attend(q[lead:lead + total], [(b, list(range(n - t, n))) for b, (n, t) in enumerate(zip(c.lens, new))],
                        lambda b, g, p: visible(c.lens[b], p, window, sinks), 2.0 ** -11 if c.q4 else U)
    near(out[lead:lead + total], ref, tol)
    assert torch.all(out[:lead] == 7.0) and torch.all(out[lead + total:] == 7.0)
    assert c.ws.status() == 0
    return out


LENS = [300, 1, 0, 77, 1000, 129]


# ------------------------------------------------------------- one token each
@pytest.mark.parametrize("q4", [False, True])
@pytest.mark.parametrize("G", [1, 2, 4, 8])
@pytest.mark.parametrize("page", [0, 16, 48])
def test_token_all_positions(G, page, q4):
    run_tokens(Case(G + page, LENS, G, 2, page, q4), 0, 0)


@pytest.mark.parametrize("q4", [False, True])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 3), (16, 0), (63, 1), (128, 4), (129, 40), (999, 1), (1000, 5),
                                          (5000, 2), (200, 800), (200, 2000)])
def test_token_windows(window, sinks, q4):
    run_tokens(Case(window + sinks, LENS, 4, 1, 32, q4), window, sinks)


@pytest.mark.parametrize("q4", [False, True])
@pytest.mark.parametrize("page", [1, 5, 8, 100, 1024])
def test_token_pages(page, q4):
    run_tokens(Case(page, [513, 30, 256], 2, 3, page, q4), 200, 7)


@pytest.mark.parametrize("q4", [False, True])
@pytest.mark.parametrize("B,N,Hkv", [(1, 20000, 1), (300, 40, 2), (3, 4100, 8)])
def test_token_splits(B, N, Hkv, q4):
    """One long request over every SM; many short ones in one CTA's range."""
    gen = torch.Generator().manual_seed(N)
    lens = torch.randint(N // 2, N + 1, (B,), generator=gen).tolist()
    c = Case(N, lens, 8 if B < 300 else 1, Hkv, 0, q4)
    a = run_tokens(c, 0, 0)
    assert torch.equal(run_tokens(c, 0, 0).isnan(), a.isnan())


@pytest.mark.parametrize("page", [0, 16])
@pytest.mark.parametrize("k", [1, 16, 33, 500])
@pytest.mark.parametrize("G", [1, 4, 8])
def test_q4_sparse(G, k, page):
    c = Case(k + page, LENS, G, 2, page, True)
    idx = torch.full((c.B, c.Hkv, k), -1, dtype=torch.int32)
    for b, n in enumerate(c.lens):
        for g in range(c.Hkv):
            m = min(n, k - g if k > 1 else k)        # rows with and without padding
            idx[b, g, :m] = torch.randperm(max(n, 1), generator=c.gen)[:m].to(torch.int32)
            idx[b, g] = idx[b, g, torch.randperm(k, generator=c.gen)]
    q = 2 * c.rnd(c.B, G * c.Hkv, D)
    out = torch.full_like(q, 7.0).cuda()
    td.td_q4_sparse_attn(c.shape, c.cache, q.cuda(), c.seq, idx.cuda(), k, out, c.ws)
    ref, tol = c.attend(q, [(b, [n - 1]) for b, n in enumerate(c.lens)],
                        lambda b, g, p: [int(j) for j in idx[b, g] if j >= 0], 2.0 ** -11)
    near(out, ref, tol)
    assert c.ws.status() == 0
    # entries that are no positions are skipped and reported
    bad = idx.clone()
    bad[:, :, 0] = torch.tensor([-2, 1 << 30, 1000, 77, -2147483648, 129])[:, None]
    td.td_q4_sparse_attn(c.shape, c.cache, q.cuda(), c.seq, bad.cuda(), k, out, c.ws)
    bad[:, :, 0] = -1
    ref, tol = c.attend(q, [(b, [n - 1]) for b, n in enumerate(c.lens)],
                        lambda b, g, p: [int(j) for j in bad[b, g] if j >= 0], 2.0 ** -11)
    near(out, ref, tol)
    assert c.ws.status() == td.FLAG_INDEX_OUT_OF_RANGE


# ------------------------------------------------------------- many new tokens
@pytest.mark.parametrize("q4", [False, True])
@pytest.mark.parametrize("G", [1, 2, 4, 8])
@pytest.mark.parametrize("page", [0, 16, 48])
def test_new_tokens(G, page, q4):
    run_new(Case(G * 7 + page, [300, 1, 0, 77, 700, 129], G, 2, page, q4), [300, 1, 0, 5, 33, 64], 0, 0, tail=3, lead=2)


@pytest.mark.parametrize("q4", [False, True])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 2), (17, 0), (64, 1), (127, 130), (128, 4), (129, 3), (300, 300),
                                          (500, 1)])
def test_new_windows(window, sinks, q4):
    run_new(Case(window * 3 + sinks, [513, 700, 130], 2, 1, 32, q4), [513, 100, 1], window, sinks)


@pytest.mark.parametrize("q4", [False, True])
@pytest.mark.parametrize("n", [1, 2, 15, 127, 128, 129, 255, 256, 257, 385])
def test_new_lengths_around_tiles(n, q4):
    run_new(Case(n, [n, n + 128], 1, 1, 16, q4), [n, n], 0, 0)
    run_new(Case(n, [n, n + 40], 8, 1, 0, q4), [n, n], 100, 2)


@pytest.mark.parametrize("q4", [False, True])
def test_new_many_requests(q4):
    lens = [1 + (i * 37) % 90 for i in range(70)]
    run_new(Case(5, lens, 4, 2, 8, q4), [min(n, 1 + (i * 13) % 40) if i % 9 else 0 for i, n in enumerate(lens)], 30, 2)


@pytest.mark.parametrize("q4", [False, True])
@pytest.mark.parametrize("G,new,window", [(1, [3, 0], 0), (4, [70, 9], 0), (8, [5, 40], 3001), (2, [200, 131], 0)])
def test_few_new_tokens_on_long_contexts(G, new, window, q4):
    """Units of many times a CTA's share: every one is cut often."""
    run_new(Case(sum(new) + G, [5003, 4100], G, 1, 48, q4), new, window, 3)


def test_forms_agree():
    """One token per request through both forms."""
    c = Case(9, [700, 129, 64], 4, 2, 16)
    q = c.rnd(3, 8, D).cuda()
    a, b = torch.zeros_like(q), torch.zeros_like(q)
    td.td_window_attn(c.shape, c.cache, 300, 4, None, q, c.seq, a, c.ws)
    td.td_window_attn(c.shape, c.cache, 300, 4, i32([0, 1, 2, 3]), q, c.seq, b, c.ws)
    assert (a.float() - b.float()).abs().max().item() < 2e-2


@pytest.mark.parametrize("q4", [False, True])
def test_hidden_values_do_not_reach_rows(q4):
    """Values that are not finite at positions that some rows of a unit see and others do not."""
    c = Case(3, [400, 300], 2, 1, 0, q4)
    if q4:
        for pos, what in ((390, 8), (150, 8), (151, 0)):
            c.parts[2][0, 0, pos, what] = 0x7f
        c.V[0, 0, [390, 150], :16] = float("nan")
        c.K[0, 0, 151, :16] = float("nan")
    else:
        for x, pos in ((c.V, 390), (c.V, 150), (c.K, 151)):
            x[0, 0, pos, :5] = float("nan")
        c.V[0, 0, 392, 7] = float("inf")
        c.parts[0].copy_(c.K), c.parts[1].copy_(c.V)
    q = 2 * c.rnd(160, 2, D)
    out = torch.zeros_like(q).cuda()
    call(c)(c.shape, c.cache, 64, 2, i32([0, 100, 160]), q.cuda(), c.seq, out, c.ws)
    K, V = c.K.clone(), c.V.clone()
    for i in range(160):
        b, p = (0, 300 + i) if i < 100 else (1, 140 + i)
        pos = visible(c.lens[b], p, 64, 2)
        z = q[i].double() @ K[b, 0, pos].double().T / D ** 0.5
        want = torch.softmax(z, -1) @ V[b, 0, pos].double()
        got = out[i].cpu().double()
        assert torch.equal(got.isfinite(), want.isfinite()), (i, p)
        fine = want.isfinite()
        assert (got - want)[fine].abs().max().item() <= 3e-2 if fine.any() else True


@pytest.mark.parametrize("q4", [False, True])
@pytest.mark.parametrize("kind", ["up", "down", "waves", "cliff", "last"])
def test_scores_that_rise_and_fall(kind, q4):
    """Scores whose maximum moves by far more than the running one may lag, within and between tiles."""
    n = 700
    c = Case(17, [n], 4, 1, 0, q4)
    j = torch.arange(n).float()
    slope = {"up": j / 4, "down": -j / 4, "waves": 90 * torch.sin(j / 40), "cliff": torch.where(j < 200, -400.0, 0.0),
             "last": torch.where(j < n - 1, 0.0, 150.0)}[kind]
    w = torch.sign(c.rnd(D).float())
    K = (c.K.float() + (slope[:, None] * w * D ** 0.5 / D)).to(torch.bfloat16)       # score: about the slope
    if q4:
        codes, scales = quantise(K)
        c.K = values(codes, scales)
        c.parts[0].copy_(codes), c.parts[2][..., :8].copy_(scales)
    else:
        c.K = K
        c.parts[0].copy_(K)
    plain = c.rnd
    c.rnd = lambda *s: ((plain(*s).float() / 4 + w) / 2).to(torch.bfloat16)          # (they double it)
    run_new(c, [n], 0, 0)
    run_new(c, [330], 200, 3)
    run_tokens(c, 0, 0)
    run_tokens(c, 300, 2)


def test_more_new_tokens_than_cached():
    c = Case(4, [5, 40], 4, 2, 0)
    q = c.rnd(30, 8, D).cuda()
    out = torch.full_like(q, 7.0)
    td.td_window_attn(c.shape, c.cache, 8, 1, i32([0, 20, 30]), q, c.seq, out, c.ws)
    assert c.ws.status() == td.FLAG_SEQ_LEN_OUT_OF_RANGE
    assert torch.all(out[:15] == 0.0) and not out.isnan().any()
    ref, tol = c.attend(q.cpu()[15:], [(0, list(range(5))), (1, list(range(30, 40)))],
                        lambda b, g, p: visible(c.lens[b], p, 8, 1), U)
    near(out[15:], ref, tol)


@pytest.mark.parametrize("q4", [False, True])
def test_pages_that_are_none(q4):
    """Their tokens are skipped and reported, in every form."""
    c = Case(6, [200, 333], 4, 2, 16, q4)
    c.dev_table[0, 3], c.dev_table[1, 20] = -1, c.pages
    gone = {0: range(48, 64), 1: range(320, 333)}
    see = lambda b, g, p: [j for j in visible(c.lens[b], p, 150, 60) if j not in gone[b]]
    q = 2 * c.rnd(60, 8, D)
    out = torch.zeros_like(q).cuda()
    call(c)(c.shape, c.cache, 150, 60, i32([0, 20, 60]), q.cuda(), c.seq, out, c.ws)
    ref, tol = c.attend(q, [(0, list(range(180, 200))), (1, list(range(293, 333)))], see, 2.0 ** -11 if q4 else U)
    near(out, ref, tol)
    assert c.ws.status() == td.FLAG_PAGE_OUT_OF_RANGE
    q = q[:2]
    out = torch.zeros_like(q).cuda()
    call(c)(c.shape, c.cache, 150, 60, None, q.cuda(), c.seq, out, c.ws)
    ref, tol = c.attend(q, [(0, [199]), (1, [332])], see, 2.0 ** -11 if q4 else U * U)
    near(out, ref, tol)
    assert c.ws.status() == td.FLAG_PAGE_OUT_OF_RANGE


def test_lengths_out_of_range_are_clamped():
    c = Case(8, [50, 50], 1, 1, 0)
    c.seq.copy_(i32([51, -3]))
    q = c.rnd(2, 1, D)
    out = torch.zeros_like(q).cuda()
    td.td_window_attn(c.shape, c.cache, 0, 0, None, q.cuda(), c.seq, out, c.ws)
    assert c.ws.status() == td.FLAG_SEQ_LEN_OUT_OF_RANGE
    ref, tol = c.attend(q, [(0, [49]), (1, [-1])], lambda b, g, p: visible(50, p, 0, 0), U * U)
    near(out, ref, tol)


def test_q_of_any_size_over_4_bits():
    """q rows from 2^-126 to 2^127 keep their direction in fp16."""
    c = Case(12, [64], 8, 1, 0, True)
    q = c.rnd(1, 8, D)
    for h, e in enumerate([-120, -60, -20, 0, 3, 5, 6, 7]):
        q[0, h] = (q[0, h].double() * 2.0 ** e).to(torch.bfloat16)
    for cu in (None, i32([0, 1])):
        out = torch.zeros_like(q).cuda()
        td.td_q4_attn(c.shape, c.cache, 0, 0, cu, q.cuda(), c.seq, out, c.ws)
        ref, tol = c.attend(q, [(0, [63])], lambda b, g, p: range(64), 2.0 ** -11)
        near(out, ref, tol)


# ------------------------------------------------------------- append
@pytest.mark.parametrize("Hkv,page,tokens", [(1, 1, 7), (2, 16, 61), (8, 48, 500), (3, 7, 1)])
def test_q4_append(Hkv, page, tokens):
    gen = torch.Generator().manual_seed(tokens)
    pages = -(-tokens // page) + 3
    wide = torch.randn(tokens, 2 * Hkv * D + 16, generator=gen)
    wide *= torch.exp(3 * torch.randn(tokens, 1, generator=gen))
    wide[tokens // 2] *= 1e-3                                          # scales below e4m3's smallest
    # every border between two codes, and values right beside it
    rule = torch.tensor([6, .25, .75, 1.25, 1.75, 2.5, 3.5, 5, -.25, -.75, -1.25, -5, 0, -0., .2490234375, 4.96875])
    wide[0, :16] = rule * 1.75
    wide = wide.to(torch.bfloat16)
    k, v = wide[:, 8:8 + Hkv * D].view(tokens, Hkv, D), wide[:, 8 + Hkv * D:8 + 2 * Hkv * D].view(tokens, Hkv, D)
    slots = torch.randperm(pages * page, generator=gen)[:tokens].to(torch.int32)
    if tokens > 4:
        slots[2], slots[3] = -1, pages * page
    dims = (pages, Hkv, page)
    codes = [torch.full(dims + (64,), 0xaa, dtype=torch.uint8).cuda() for _ in range(2)]
    scales = torch.full(dims + (16,), 0x55, dtype=torch.uint8).cuda()
    want = [x.cpu().clone() for x in codes + [scales]]
    dev = wide.cuda()
    kd = dev[:, 8:8 + Hkv * D].view(tokens, Hkv, D)
    vd = dev[:, 8 + Hkv * D:8 + 2 * Hkv * D].view(tokens, Hkv, D)
    td.td_q4_append(td.make_shape(1, Hkv, Hkv, 16), td.make_q4_cache(*codes, scales), kd, vd, slots.cuda())
    (kc, ks), (vc, vs) = quantise(k), quantise(v)
    for i, s in enumerate(slots.tolist()):
        if 0 <= s < pages * page:
            at = (s // page, slice(None), s % page)
            want[0][at], want[1][at], want[2][at] = kc[i], vc[i], torch.cat([ks[i], vs[i]], -1)
    for got, ref in zip(codes + [scales], want):
        assert (got.cpu() != ref).sum().item() == 0


def test_q4_append_values_out_of_range():
    x = torch.randn(6, 1, D).to(torch.bfloat16)
    x[0, 0, 3], x[1, 0, 20], x[2, 0, 40] = float("nan"), float("inf"), -float("inf")
    x[3, 0, 0:16], x[4], x[5] = 3e38, 0.0, 1e-30
    codes = [torch.zeros(6, 1, 1, 64, dtype=torch.uint8).cuda() for _ in range(2)]
    scales = torch.zeros(6, 1, 1, 16, dtype=torch.uint8).cuda()
    td.td_q4_append(td.make_shape(1, 1, 1, 1), td.make_q4_cache(*codes, scales), x.cuda(), x.cuda(),
                    torch.arange(6, dtype=torch.int32).cuda())
    c, s = quantise(x)
    assert torch.equal(scales.cpu()[:, 0, 0, :8], s[:, 0]) and torch.equal(scales.cpu()[:, 0, 0, 8:], s[:, 0])
    assert torch.equal(codes[0].cpu()[:, 0, 0], c[:, 0]) and torch.equal(codes[1].cpu()[:, 0, 0], c[:, 0])


def test_q4_append_every_short_number():
    """All positive bf16 values between 2^-12 and 2^12 against every scale that their block can have."""
    bits = torch.arange((127 - 12) << 7, (127 + 12) << 7, dtype=torch.int32).to(torch.int16)
    x = bits.view(torch.bfloat16)
    rows = []
    for top in (6.0, 6.5, 7.75, 100.0, 3.0, 2688.0, 0.02):
        y = x[x <= top]
        y = torch.cat([y, y.new_full((-len(y) % 15,), 0.0)]).view(-1, 15)
        rows.append(torch.cat([y.new_full((len(y), 1), top), y], 1))
    x = torch.cat(rows)
    x = torch.cat([x, x.new_zeros(-len(x) % 8, 16)]).view(-1, 1, D)
    n = len(x)
    codes = [torch.zeros(n, 1, 1, 64, dtype=torch.uint8).cuda() for _ in range(2)]
    scales = torch.zeros(n, 1, 1, 16, dtype=torch.uint8).cuda()
    td.td_q4_append(td.make_shape(1, 1, 1, 1), td.make_q4_cache(*codes, scales), x.cuda(), (-x).cuda(),
                    torch.arange(n, dtype=torch.int32).cuda())
    for c, sign, at in ((codes[0], 1, slice(0, 8)), (codes[1], -1, slice(8, 16))):
        want, s = quantise(sign * x)
        assert torch.equal(scales.cpu()[:, 0, 0, at], s[:, 0]) and torch.equal(c.cpu()[:, 0, 0], want[:, 0])


# ------------------------------------------------------------- weights
@pytest.mark.parametrize("G", [1, 2, 4, 8])
@pytest.mark.parametrize("page,fresh", [(0, 1), (16, 0), (48, 64), (0, 5000)])
def test_weights(G, page, fresh):
    c = Case(G + page, LENS, G, 2, page)
    q = 2 * c.rnd(c.B, G * c.Hkv, D)
    old = torch.rand(c.B, c.Hkv, c.N, generator=c.gen)
    w, logits = old.cuda(), torch.full((c.B, G * c.Hkv, c.N), 9.0).cuda()
    out = torch.full_like(q, 7.0).cuda()
    td.td_weights_attn(c.shape, c.cache, fresh, q.cuda(), c.seq, w, logits, out, c.ws)
    ref, tol = c.attend(q, [(b, [n - 1]) for b, n in enumerate(c.lens)], lambda b, g, p: range(c.lens[b]), U * U)
    near(out, ref, tol)
    for b, n in enumerate(c.lens):
        assert torch.all(logits[b, :, n:] == 9.0) and torch.equal(w[b, :, n:].cpu(), old[b, :, n:])
        for g in range(c.Hkv):
            keep = torch.where(torch.arange(n) < n - fresh, old[b, g, :n].double(), 0.0)
            want, err = keep.clone(), torch.zeros(n, dtype=torch.float64)
            for h in range(g * G, (g + 1) * G):
                K, V = c.K[b, g, :n].double(), c.V[b, g, :n].double()
                _, _, a, rel = attend(q[b:b + 1, h], K, V, torch.ones(1, n, dtype=torch.bool), 0.0)
                want += a[0]
                err += a[0] * rel[0]
                z = (K @ q[b, h].double()) / D ** 0.5
                bound = D * E * ((K.abs() @ q[b, h].double().abs()) / D ** 0.5) + 2 * E * z.abs()
                near(logits[b, h, :n], z, bound)
            near(w[b, g, :n], want, err + (G + 1) * E * want)
    assert c.ws.status() == 0


# ------------------------------------------------------------- eviction
def run_evict(c, w, budget, sinks, recent, place, to_page=0, row=None):
    to_n = min(budget, c.N)
    old_k, old_v = c.parts[0].clone(), c.parts[1].clone()
    wd = w.cuda()
    if place:
        to, tk, tv, wo, tt, page = c.cache, c.parts[0], c.parts[1], wd, c.table, c.page
    else:
        page = to_page
        if page:
            blocks = -(-to_n // page)
            tt = torch.randperm(c.B * blocks + 2, generator=c.gen)[:c.B * blocks].view(c.B, blocks).to(torch.int32)
            dims = (c.B * blocks + 2, c.Hkv, page, D)
        else:
            tt, dims = None, (c.B, c.Hkv, to_n, D)
        tk, tv = (torch.full(dims, 5.0, dtype=torch.bfloat16).cuda() for _ in range(2))
        to = td.make_cache(tk, tv, None if tt is None else tt.cuda())
        wo = torch.full((c.B, c.Hkv, row or to_n), 3.0).cuda()
    before = [tk.cpu().clone(), tv.cpu().clone(), wo.cpu().clone()]
    kept = torch.full((c.B, c.Hkv, budget), -7, dtype=torch.int32).cuda()
    seq_out = torch.zeros(c.B, dtype=torch.int32).cuda()
    td.td_evict(c.shape, c.cache, to, budget, sinks, recent, wd, wo, c.seq, seq_out, kept, c.ws)
    assert c.ws.status() == 0
    want = before
    for b, n in enumerate(c.lens):
        assert seq_out[b].item() == min(n, budget)
        for g in range(c.Hkv):
            keep = evict(w[b, g].tolist(), n, budget, sinks, recent)
            assert kept[b, g].tolist() == keep + [-1] * (budget - len(keep))
            for i, p in enumerate(keep):
                src = (b, g, p) if c.table is None else (c.table[b, p // c.page], g, p % c.page)
                dst = (b, g, i) if tt is None else (tt[b, i // page], g, i % page)
                want[0][dst], want[1][dst], want[2][b, g, i] = old_k[src].cpu(), old_v[src].cpu(), w[b, g, p]
    for got, ref in zip((tk, tv, wo), want):
        assert torch.equal(got.cpu().nan_to_num(), ref.nan_to_num())


@pytest.mark.parametrize("page", [0, 16, 48])
@pytest.mark.parametrize("budget,sinks,recent", [(1, 0, 0), (1, 0, 1), (1, 1, 0), (64, 4, 16), (77, 0, 77), (128, 100, 0),
                                                 (300, 4, 200), (999, 3, 5), (2000, 1, 1)])
@pytest.mark.parametrize("place", [True, False])
def test_evict(place, budget, sinks, recent, page):
    c = Case(budget + page, LENS, 1, 2, page)
    run_evict(c, torch.rand(c.B, c.Hkv, c.N, generator=c.gen), budget, sinks, recent, place, 32 if page else 0, None if
              budget % 2 else budget + 5)


@pytest.mark.parametrize("kind", ["equal", "few", "special", "heavy end", "close"])
@pytest.mark.parametrize("place,n", [(True, 700), (False, 700), (True, 9000), (True, 17000)])
def test_evict_weights(place, n, kind):
    """The rows' three ways through the selection, by their length."""
    c = Case(11, [n, 650, 64], 1, 2, 16)
    w = torch.rand(c.B, c.Hkv, c.N, generator=c.gen)
    if kind == "equal":
        w = torch.full_like(w, 0.25)
    elif kind == "few":
        w = (w * 4).floor()
    elif kind == "special":
        pool = torch.tensor([0.0, -0.0, float("inf"), -float("inf"), float("nan"), 1e-45, -1e-45, 1.0, -1.0])
        w = pool[(w * 9).long().clamp(max=8)]
    elif kind == "heavy end":
        w = torch.arange(c.N).float().expand_as(w).clone()
    elif kind == "close":
        w = (torch.full_like(w, 1.0).view(torch.int32) + (w * 300).int()).view(torch.float32)
    run_evict(c, w, 130, 3, 20, place)


def test_evict_many_requests_and_long_rows():
    c = Case(2, [1 + (i * 31) % 100 for i in range(40)], 1, 8, 8)
    run_evict(c, torch.rand(c.B, c.Hkv, c.N, generator=c.gen), 33, 2, 8, True)
    for n, budget in ((9000, 5000), (17000, 3), (16385, 16384)):
        c = Case(2, [n], 1, 1, 0)
        run_evict(c, (torch.rand(1, 1, c.N, generator=c.gen) * 5000).floor(), budget, 1, 2, True)


@pytest.mark.parametrize("few", [False, True])
@pytest.mark.parametrize("B,Hkv,N", [(10, 8, 3000), (11, 8, 8193), (3, 1, 2049), (7, 8, 16384), (10, 8, 9000),
                                     (2, 8, 4097), (1, 2, 16385), (2, 1, 131072), (1, 1, 131073)])
def test_evict_selection_of_many_and_of_long_rows(B, Hkv, N, few):
    """Every way through the selection: rows few and many, up to where each way ends."""
    gen = torch.Generator(device="cuda").manual_seed(N)
    shape = td.make_shape(B, Hkv, Hkv, N)
    k = torch.zeros(B, Hkv, N, D, dtype=torch.bfloat16, device="cuda")
    at = torch.arange(N, device="cuda")
    for i, x in enumerate((at // 65536, at // 256 % 256, at % 256)):
        k[..., i] = x                                           # (exact in bf16)
    budget, sinks, recent = N // 3, 5, N // 7
    to = torch.full((B, Hkv, budget, D), 9.0, dtype=torch.bfloat16, device="cuda")
    w = torch.rand(B, Hkv, N, generator=gen, device="cuda")
    if few:
        w = (w * 5).floor()
    lens = i32([N - 17 * b for b in range(B)])
    out, kept = torch.zeros(B, Hkv, budget).cuda(), torch.zeros(B, Hkv, budget, dtype=torch.int32).cuda()
    seq, ws = i32([0] * B), td.Workspace(shape, 0, cache_calls=True)
    td.td_evict(shape, td.make_cache(k, k), td.make_cache(to, to.clone()), budget, sinks, recent, w, out, lens, seq, kept, ws)
    fixed = (at < sinks) | (at >= lens[:, None] - recent)
    key = torch.where(fixed[:, None], 9.0, w).where(at < lens[:, None, None], -1.0)
    want = key.sort(dim=-1, descending=True, stable=True).indices[..., :budget].sort(dim=-1).values
    assert torch.equal(kept.long(), want) and torch.equal(out, w.gather(-1, want))
    rows = (to[..., :3].float() * torch.tensor([65536.0, 256.0, 1.0], device="cuda")).sum(-1)
    assert torch.equal(rows.long(), want) and ws.status() == 0
    assert seq.tolist() == [budget] * B


def test_evict_pages_that_are_none():
    c = Case(6, [200], 1, 1, 16)
    c.dev_table[0, 3] = -1
    old = c.parts[0].clone()
    w = torch.arange(200).float().view(1, 1, 200).cuda()
    kept = torch.zeros(1, 1, 150, dtype=torch.int32).cuda()
    out = torch.zeros(1, dtype=torch.int32).cuda()
    td.td_evict(c.shape, c.cache, c.cache, 150, 0, 0, w, w, c.seq, out, kept, c.ws)
    assert kept[0, 0].tolist() == list(range(50, 200)) and c.ws.status() == td.FLAG_PAGE_OUT_OF_RANGE
    at = lambda p: (int(c.table[0, p // 16]), 0, p % 16)
    for i in range(150):
        src = i if i // 16 == 3 or (i + 50) // 16 == 3 else i + 50
        if i // 16 != 3:
            assert torch.equal(c.parts[0][at(i)].cpu().nan_to_num(), old[at(src)].cpu().nan_to_num()), i


# ------------------------------------------------------------- far rows
@pytest.mark.parametrize("q4", [False, True])
def test_offsets_beyond_32_bits(q4):
    N = (1 << 26 if q4 else 1 << 24) + 300        # rows of 64 or 256 bytes: beyond 4 GB
    shape = td.make_shape(1, 4, 1, N)
    gen = torch.Generator().manual_seed(1)
    x = [torch.randn(1, 1, 400, D, generator=gen).to(torch.bfloat16) for _ in range(2)]
    if q4:
        (kc, ks), (vc, vs) = quantise(x[0]), quantise(x[1])
        parts = [torch.zeros(1, 1, N, w, dtype=torch.uint8, device="cuda") for w in (64, 64, 16)]
        for p, y in zip(parts, (kc, vc, torch.cat([ks, vs], -1))):
            p[:, :, -400:] = y.cuda()
        K, V = values(kc, ks), values(vc, vs)
        cache = td.make_q4_cache(*parts)
    else:
        parts = [torch.zeros(1, 1, N, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        for p, y in zip(parts, x):
            p[:, :, -400:] = y.cuda()
        K, V = x
        cache = td.make_cache(*parts)
    ws = td.Workspace(shape, 0, cache_calls=True)
    fn = td.td_q4_attn if q4 else td.td_window_attn
    for T, cu in ((1, None), (50, i32([0, 50]))):
        q = 2 * torch.randn(T, 4, D, generator=gen).to(torch.bfloat16)
        out = torch.zeros_like(q).cuda()
        fn(shape, cache, 200, 0, cu, q.cuda(), i32([N]), out, ws)
        sees = torch.zeros(T, 400, dtype=torch.bool)
        for t in range(T):
            sees[t, 400 - T + t + 1 - 200:400 - T + t + 1] = True
        for h in range(4):
            ref, tol, _, _ = attend(q[:, h], K[0, 0].double(), V[0, 0].double(), sees, 2.0 ** -11 if q4 else U, q4)
            near(out[:, h], ref, tol)
    assert ws.status() == 0
