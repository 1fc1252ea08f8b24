"""Eviction where the rows' moves take several lists of positions, the selection keeps first and last positions
alone, and the kept rows go to pages of the same pool."""
import pytest
import torch

import sparse_attention_td_gb300 as td
from cache_util import D
from test_cache_gpu import _built, i32  # noqa: F401

pytestmark = pytest.mark.gpu


class Numbered:
    """Requests whose rows hold their own numbers (exact in bf16), those of V the other way round."""

    def __init__(self, lens, Hkv, N, page=0, spare=0):
        self.lens, self.B, self.Hkv, self.N, self.page = lens, len(lens), Hkv, N, page
        self.shape = td.make_shape(self.B, Hkv, Hkv, N)
        self.table = None
        dims, at = (self.B, Hkv, N), torch.arange(N, device="cuda").expand(self.B, Hkv, N)
        if page:
            blocks = -(-N // page)
            dims = (self.B * blocks + spare, Hkv, page)
            gen = torch.Generator().manual_seed(N)
            order = torch.randperm(dims[0], generator=gen).cuda()
            self.table = order[:self.B * blocks].view(self.B, blocks).to(torch.int32)
            self.spare = order[self.B * blocks:].to(torch.int32)
            at = torch.full((dims[0], page), -1, device="cuda")
            at[self.table.long()] = torch.arange(blocks * page, device="cuda").view(blocks, page).expand(self.B, -1, -1)
            at = at[:, None].expand(dims)
        self.k, self.v = (torch.zeros(*dims, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        self.write(self.k, at)
        self.write(self.v, (1 << 23) - at)
        self.cache = td.make_cache(self.k, self.v, self.table)
        self.seq = i32(lens)
        self.seq_out = i32([0] * self.B)
        self.ws = td.Workspace(self.shape, 0, cache_calls=True)

    @staticmethod
    def write(x, at):
        head = torch.arange(at.shape[1], device="cuda")[:, None].expand(at.shape)
        for lane in (0, 48, 80, 112):                  # (a number in every slice of a row)
            for i, part in enumerate((at // 65536, at // 256 % 256, at % 256, head)):
                x[..., lane + i] = part.to(torch.bfloat16)

    def numbers(self, x, table=None):
        """The numbers in the rows of every request, [B][Hkv][positions]; each slice has to hold the same."""
        if table is not None:
            x = x[table.long()].transpose(1, 2).flatten(2, 3)
        parts = [(x[..., i:i + 3].float() * torch.tensor([65536.0, 256.0, 1.0], device="cuda")).sum(-1).long()
                 for i in (0, 48, 80, 112)]
        assert all(torch.equal(parts[0], p) for p in parts[1:])
        assert torch.equal(x[..., 3].long(), torch.arange(self.Hkv, device="cuda")[:, None].expand(x.shape[:3]))
        return parts[0]

    def evict(self, to, w, budget, sinks, recent, out=None):
        kept = torch.full((self.B, self.Hkv, budget), -7, dtype=torch.int32, device="cuda")
        td.td_evict(self.shape, self.cache, to, budget, sinks, recent, w, w if out is None else out, self.seq,
                    self.seq_out, kept, self.ws)
        assert self.ws.status() == 0
        assert self.seq_out.tolist() == [min(n, budget) for n in self.lens]
        return kept.long()

    def wanted(self, w, budget, sinks, recent):
        """The kept positions, ascending, -1 padded."""
        at, n = torch.arange(self.N, device="cuda"), torch.tensor(self.lens, device="cuda")[:, None, None]
        fixed = (at < sinks) | (at >= n - recent)
        key = torch.where(fixed, 9.0, w).where(at < n, -1.0)
        some = min(budget, self.N)
        want = key.sort(dim=-1, descending=True, stable=True).indices[..., :some]
        want = torch.where(want < n, want, 1 << 30).sort(dim=-1).values
        want = torch.where(n <= budget, torch.arange(some, device="cuda"), want)
        want = torch.where(want < n, want, -1)
        return torch.nn.functional.pad(want, (0, budget - some), value=-1)

    def check_rows(self, k, v, want, table=None):
        k, v = self.numbers(k, table), self.numbers(v, table)
        there = want >= 0
        assert torch.equal(k[..., :want.shape[-1]][there], want[there])
        assert torch.equal(v[..., :want.shape[-1]][there], (1 << 23) - want[there])


@pytest.mark.parametrize("page", [0, 64])
@pytest.mark.parametrize("budget", [1025, 2500, 5000])
def test_one_late_position_leaves_a_long_cache(budget, page):
    """In place, as a decode step does it: every list of rows but the last one stays where it is."""
    lens, n = [budget + 1, budget, budget + 1, 700], budget + 1
    gone = budget - 40                                 # (in the last list of 1024, or near its begin)
    for _ in range(10):
        c = Numbered(lens, 2, n, page)
        w = torch.rand(4, 2, n, device="cuda") + 0.5
        w[:, :, gone] = 0.25
        want = c.wanted(w, budget, 4, 20)
        assert want[0, 0, gone - 1:gone + 1].tolist() == [gone - 1, gone + 1]
        kept = c.evict(c.cache, w, budget, 4, 20)
        assert torch.equal(kept, want)
        c.check_rows(c.k, c.v, want, c.table)


def test_many_requests_with_several_lists_each():
    """Between two caches, more rows than CTAs can be cut for: each walks over lists of its own."""
    c = Numbered([2100 - 3 * (b % 17) for b in range(80)], 8, 2100)
    budget = 2050
    w = torch.rand(c.B, c.Hkv, c.N, device="cuda")
    want = c.wanted(w, budget, 3, 100)
    for _ in range(5):
        k, v = (torch.zeros(c.B, c.Hkv, budget, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        for x in (k, v):
            c.write(x, torch.full(x.shape[:3], -1, device="cuda"))
        kept = c.evict(td.make_cache(k, v), w, budget, 3, 100, torch.zeros(c.B, c.Hkv, budget, device="cuda"))
        assert torch.equal(kept, want)
        c.check_rows(k, v, want)


@pytest.mark.parametrize("place", [True, False])
@pytest.mark.parametrize("B,N", [(3, 1000), (2, 4097), (40, 9000), (2, 16385), (1, 131072), (1, 131073)])
def test_first_and_last_positions_alone(B, N, place):
    """budget = sinks + recent: no weight decides, on every way through the selection."""
    c = Numbered([N - 7 * b for b in range(B)], 2, N)
    budget, sinks = 700, 11
    w = torch.rand(B, 2, N, device="cuda")
    want, old = c.wanted(w, budget, sinks, budget - sinks), w.clone()
    for b, n in enumerate(c.lens):
        assert want[b, 0].tolist() == list(range(sinks)) + list(range(n - budget + sinks, n))
    if place:
        k, v, out = c.k, c.v, w
        kept = c.evict(c.cache, w, budget, sinks, budget - sinks)
    else:
        k, v = (torch.zeros(B, 2, budget, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        out = torch.zeros(B, 2, budget, device="cuda")
        kept = c.evict(td.make_cache(k, v), w, budget, sinks, budget - sinks, out)
    assert torch.equal(kept, want) and torch.equal(out[..., :budget], old.gather(-1, want))
    c.check_rows(k, v, want)


@pytest.mark.parametrize("blocks", ["same", "some", "other"])
@pytest.mark.parametrize("B,N,page,budget", [(3, 600, 16, 100), (2, 5000, 64, 2500), (1, 9000, 48, 1025), (60, 300, 8, 64)])
def test_two_tables_of_one_pool(B, N, page, budget, blocks):
    """The kept rows go by a shorter copy of the cache's table, by pages of their own, or some of each."""
    need = -(-budget // page)
    lens = [N - 11 * (b % 20) if b % 3 < 2 else budget - b for b in range(B)]      # (some keep all they have)
    c = Numbered(lens, 2, N, page, spare=B * need)
    spare = c.spare.view(B, need)
    table = c.table[:, :need].clone()
    if blocks == "other":
        table = spare.clone()
    elif blocks == "some":
        pick = torch.rand(B, need, device="cuda") < 0.5
        pick[0] = True                                                       # (a request with none of its own)
        table = torch.where(pick, spare, table)
    w = torch.rand(B, 2, N, device="cuda")
    want = c.wanted(w, budget, 2, 9)
    before = [x.clone() for x in (c.k, c.v)]
    out = torch.zeros(B, 2, budget, device="cuda")
    kept = c.evict(td.make_cache(c.k, c.v, table.contiguous()), w, budget, 2, 9, out)
    assert torch.equal(kept, want)
    c.check_rows(c.k, c.v, want, table)
    left = torch.ones(len(c.k), dtype=torch.bool, device="cuda")
    left[table.long().flatten()] = False
    assert torch.equal(c.k[left], before[0][left]) and torch.equal(c.v[left], before[1][left])
