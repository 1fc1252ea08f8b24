"""The entry points of the operators on small caches on the host: workspace sizes and
refusals.  Every call here fails validation or has nothing to do, so no pointer is followed
and nothing is launched."""
import ctypes

import pytest

import sparse_attention_td_gb300 as td
from sparse_attention_td_gb300 import build as libbuild
from sparse_attention_td_gb300._lib import _Cache, _Q4Cache

OK, INVALID, UNSUPPORTED, WS_SMALL = 0, 1, 2, 4
FAKE = 1 << 20
BIG = 1 << 50


@pytest.fixture(scope="module")
def L():
    libbuild.build()
    return td.lib()


def shape(batch=2, hq=8, hkv=2, n=1000, d=128, scale=0.0):
    return td.Shape(batch, hq, hkv, d, n, scale)


def cache(k=FAKE, v=1 << 40, pages=2, page=1000, table=None, blocks=0):
    return _Cache(k, v, pages, page, table, blocks)


def q4(k=FAKE, v=1 << 40, scales=1 << 45, pages=2, page=1000, table=None, blocks=0):
    return _Q4Cache(k, v, scales, pages, page, table, blocks)


def new(L, s=None, c=None, window=10, sinks=1, tokens=7, cu=FAKE, q=FAKE, seq=FAKE, out=FAKE, ws=FAKE, wsb=BIG,
        form="window"):
    s = s or shape()
    call, c = (L.td_window_attn, c or cache()) if form == "window" else (L.td_q4_attn, c or q4())
    return call(ctypes.byref(s), ctypes.byref(c), window, sinks, tokens, cu, q, seq, out, ws, wsb, None)


def test_workspace_size(L):
    n = td.td_cache_workspace_size(shape())
    assert n > 0 and td.td_cache_workspace_size(shape(batch=1000)) > n
    assert td.td_cache_workspace_size(shape(d=64)) == 0
    assert td.td_cache_workspace_size(shape(hq=6)) == 0
    assert L.td_cache_workspace_size(None) == 0


@pytest.mark.parametrize("form", ["window", "q4"])
def test_new_token_refusals(L, form):
    f = lambda **kw: new(L, form=form, **kw)
    for name in ("q", "out", "seq", "ws"):
        assert f(**{name: None}) == INVALID
    assert f(q=FAKE + 8) == INVALID and f(out=FAKE + 2) == INVALID
    assert f(seq=FAKE + 2) == INVALID and f(cu=FAKE + 1) == INVALID and f(ws=FAKE + 128) == INVALID
    assert f(window=-1) == INVALID and f(sinks=-1) == INVALID and f(tokens=-1) == INVALID
    assert f(cu=None, tokens=7) == INVALID                       # one token per request: batch of them
    assert f(wsb=td.td_cache_workspace_size(shape()) - 1) == WS_SMALL
    assert f(s=shape(d=64)) == UNSUPPORTED and f(s=shape(hq=6)) == UNSUPPORTED
    assert f(s=shape(scale=float("inf"))) == INVALID
    assert f(tokens=0, q=None, out=None) == OK                   # nothing to do
    t = q4 if form == "q4" else cache
    assert f(c=t(table=FAKE, page=16, pages=1 << 20, blocks=1 << 26), s=shape(n=(1 << 30) + 1)) == UNSUPPORTED
    assert f(s=shape(hq=2, batch=1 << 26), c=t(pages=1 << 29, page=1, table=FAKE, blocks=1000)) == UNSUPPORTED
    assert f(tokens=(1 << 31) - 1, s=shape(batch=2, hq=1024, hkv=128), c=t(pages=2)) == UNSUPPORTED


@pytest.mark.parametrize("form", ["window", "q4"])
def test_cache_refusals(L, form):
    t = q4 if form == "q4" else cache
    f = lambda **kw: new(L, form=form, c=t(**kw))
    assert f(k=None) == INVALID and f(v=None) == INVALID and f(v=FAKE + 8) == INVALID
    assert f(pages=0) == INVALID and f(page=0) == INVALID and f(pages=1) == INVALID and f(page=999) == INVALID
    assert f(page=16, table=FAKE, blocks=62) == INVALID and f(page=16, table=FAKE + 2, blocks=63) == INVALID
    assert f(pages=1 << 20, page=1 << 11) == UNSUPPORTED and f(pages=1 << 20, page=1 << 10) == UNSUPPORTED
    if form == "q4":
        assert f(scales=None) == INVALID and f(scales=FAKE + 8) == INVALID


def sparse(L, s=None, c=None, q=FAKE, seq=FAKE, idx=FAKE, k=8, out=FAKE, ws=FAKE, wsb=BIG):
    s, c = s or shape(), c or q4()
    return L.td_q4_sparse_attn(ctypes.byref(s), ctypes.byref(c), q, seq, idx, k, out, ws, wsb, None)


def test_q4_sparse_refusals(L):
    for name in ("q", "seq", "idx", "out", "ws"):
        assert sparse(L, **{name: None}) == INVALID
    assert sparse(L, idx=FAKE + 1) == INVALID and sparse(L, k=0) == INVALID and sparse(L, k=1001) == INVALID
    assert sparse(L, c=q4(page=999)) == INVALID
    assert sparse(L, wsb=1000) == WS_SMALL


def append(L, s=None, c=None, n=5, k=FAKE, v=FAKE, stride=256, slots=FAKE):
    s, c = s or shape(), c or q4()
    return L.td_q4_append(ctypes.byref(s), ctypes.byref(c), n, k, v, stride, slots, None)


def test_q4_append_refusals(L):
    assert append(L, n=-1) == INVALID
    assert append(L, k=None) == INVALID and append(L, v=FAKE + 8) == INVALID
    assert append(L, slots=None) == INVALID and append(L, slots=FAKE + 1) == INVALID
    assert append(L, stride=255) == INVALID and append(L, stride=260) == INVALID
    assert append(L, c=q4(scales=None)) == INVALID
    assert append(L, s=shape(d=64)) == UNSUPPORTED
    assert append(L, n=0, k=None, v=None, slots=None) == OK


def weights(L, s=None, c=None, fresh=1, q=FAKE, seq=FAKE, w=1 << 30, logits=1 << 35, out=FAKE, ws=FAKE, wsb=BIG):
    s, c = s or shape(), c or cache()
    return L.td_weights_attn(ctypes.byref(s), ctypes.byref(c), fresh, q, seq, w, logits, out, ws, wsb, None)


def test_weights_refusals(L):
    for name in ("q", "seq", "w", "logits", "out", "ws"):
        assert weights(L, **{name: None}) == INVALID
    assert weights(L, fresh=-1) == INVALID and weights(L, w=FAKE + 2) == INVALID
    assert weights(L, logits=(1 << 30) + 15996) == INVALID       # over the weights' last entry
    assert weights(L, wsb=1000) == WS_SMALL
    assert weights(L, c=cache(page=999)) == INVALID


EV = dict(budget=100, sinks=4, recent=10, w=1 << 30, wo=1 << 30, row=1000, seq=1 << 35, seq_out=1 << 36, kept=1 << 37,
          ws=FAKE, wsb=BIG)


def evict(L, s=None, c=None, to=None, **kw):
    a = dict(EV, **kw)
    s, c = s or shape(), c or cache()
    to = to or c
    return L.td_evict(ctypes.byref(s), ctypes.byref(c), ctypes.byref(to), a["budget"], a["sinks"], a["recent"], a["w"],
                      a["wo"], a["row"], a["seq"], a["seq_out"], a["kept"], a["ws"], a["wsb"], None)


def test_evict_refusals(L):
    for name in ("w", "wo", "seq", "seq_out", "kept", "ws"):
        assert evict(L, **{name: None}) == INVALID
        assert evict(L, **{name: EV[name] + 2}) == INVALID
    assert evict(L, budget=0) == INVALID and evict(L, sinks=-1) == INVALID and evict(L, recent=-1) == INVALID
    assert evict(L, sinks=50, recent=51) == INVALID
    assert evict(L, sinks=(1 << 31) - 1, recent=(1 << 31) - 1) == INVALID
    assert evict(L, wsb=255) == WS_SMALL
    assert evict(L, c=cache(page=999)) == INVALID
    # where the kept rows go: room for them, and no memory shared but a pool's other pages
    apart = dict(k=1 << 41, v=1 << 42)
    assert evict(L, to=cache(page=99, **apart)) == INVALID
    assert evict(L, to=cache(page=16, table=FAKE, blocks=6, **apart)) == INVALID
    assert evict(L, to=cache(k=FAKE + 16)) == INVALID
    assert evict(L, to=cache(k=1 << 41, v=(1 << 40) + 256)) == INVALID
    assert evict(L, to=cache(k=1 << 40, v=1 << 41)) == INVALID
    assert evict(L, to=cache(page=1000, table=FAKE, blocks=1)) == INVALID        # the pool of a contiguous cache
    # arrays over one another
    assert evict(L, row=999) == INVALID                          # weights in place, but of another row length
    assert evict(L, wo=(1 << 30) + 400) == INVALID
    assert evict(L, wo=1 << 31, row=99) == INVALID               # no room for the budget
    assert evict(L, seq_out=EV["seq"]) == INVALID and evict(L, seq_out=EV["seq"] + 4) == INVALID
    assert evict(L, kept=EV["w"] + 15996) == INVALID and evict(L, kept=EV["seq"] - 4) == INVALID
    assert evict(L, seq_out=EV["w"]) == INVALID
    assert evict(L, s=shape(hq=128, hkv=128, batch=1 << 18), c=cache(pages=1 << 18, page=1, table=FAKE, blocks=1000)) \
        == UNSUPPORTED
