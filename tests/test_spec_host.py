"""The speculative-decoding entry points on the host: workspace sizes and
refusals.  Every call here fails validation, so no pointer is followed and
nothing is launched."""
import ctypes

import pytest

import sparse_attention_td_gb300 as td
from sparse_attention_td_gb300 import build as libbuild
from sparse_attention_td_gb300._lib import _Cache

INVALID, UNSUPPORTED, WS_SMALL = 1, 2, 4
FAKE = 1 << 20
BIG = 1 << 50


@pytest.fixture(scope="module")
def L():
    libbuild.build()
    return td.lib()


def shape(**kw):
    base = dict(batch=2, hq=8, hkv=2, n=1000, d=128, scale=0.0)
    base.update(kw)
    return td.Shape(base["batch"], base["hq"], base["hkv"], base["d"], base["n"], base["scale"])


def cache(**kw):
    base = dict(k=FAKE, v=FAKE, pages=2, page=1000, table=None, blocks=0)
    base.update(kw)
    return _Cache(base["k"], base["v"], base["pages"], base["page"], base["table"], base["blocks"])


def tree(L, s=None, c=None, T=4, tl=FAKE, mask=FAKE, q=FAKE, seq=FAKE, out=FAKE, ws=FAKE, wsb=BIG,
         idx=None, k=0):
    s, c = s or shape(), c or cache()
    if k or idx:
        return L.td_tree_sparse_attn(ctypes.byref(s), ctypes.byref(c), T, tl, mask, q, seq, idx, k,
                                     out, ws, wsb, None)
    return L.td_tree_attn(ctypes.byref(s), ctypes.byref(c), T, tl, mask, q, seq, out, ws, wsb, None)


def test_tree_workspace_size(L):
    s = shape()
    assert td.td_tree_workspace_size(s, 1) > 0
    assert td.td_tree_workspace_size(s, 128) >= td.td_tree_workspace_size(s, 1)
    assert td.td_tree_workspace_size(s, 0) == 0
    assert td.td_tree_workspace_size(s, 129) == 0
    assert td.td_tree_workspace_size(shape(d=64), 4) == 0
    assert td.MAX_TREE == 128


def test_tree_refusals(L):
    assert tree(L, q=None) == INVALID
    assert tree(L, q=FAKE + 8) == INVALID
    assert tree(L, out=None) == INVALID
    assert tree(L, seq=None) == INVALID
    assert tree(L, tl=FAKE + 2) == INVALID
    assert tree(L, mask=FAKE + 2) == INVALID
    assert tree(L, T=0) == INVALID
    assert tree(L, T=129) == INVALID
    assert tree(L, ws=None) == INVALID
    assert tree(L, ws=FAKE + 128) == INVALID
    assert tree(L, wsb=td.td_tree_workspace_size(shape(), 4) - 1) == WS_SMALL
    assert tree(L, s=shape(d=64)) == UNSUPPORTED
    assert tree(L, s=shape(hq=6)) == UNSUPPORTED          # groups of 3
    assert tree(L, s=shape(scale=float("nan"))) == INVALID
    assert L.td_tree_attn(None, ctypes.byref(cache()), 4, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, BIG,
                          None) == INVALID
    assert L.td_tree_attn(ctypes.byref(shape()), None, 4, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, BIG,
                          None) == INVALID


def test_tree_sparse_refusals(L):
    assert tree(L, idx=FAKE, k=0) == INVALID
    assert tree(L, idx=FAKE, k=1001) == INVALID
    assert tree(L, idx=None, k=8) == INVALID
    assert tree(L, idx=FAKE + 1, k=8) == INVALID
    assert tree(L, idx=FAKE, k=8, q=None) == INVALID


def test_cache_refusals(L):
    assert tree(L, c=cache(k=None)) == INVALID
    assert tree(L, c=cache(v=FAKE + 8)) == INVALID
    assert tree(L, c=cache(pages=0)) == INVALID
    assert tree(L, c=cache(page=0)) == INVALID
    assert tree(L, c=cache(pages=1)) == INVALID                       # two requests, one page, no table
    assert tree(L, c=cache(page=999)) == INVALID                      # shorter than max_seq_len
    assert tree(L, c=cache(page=16, table=FAKE, blocks=62)) == INVALID    # 992 < 1000 positions
    assert tree(L, c=cache(page=16, table=FAKE, blocks=0)) == INVALID
    assert tree(L, c=cache(page=16, table=FAKE + 2, blocks=63)) == INVALID
    assert tree(L, c=cache(pages=1 << 20, page=1 << 11)) == UNSUPPORTED   # 2^31 slots
    assert tree(L, c=cache(pages=1 << 20, page=1 << 10)) == UNSUPPORTED   # 2^31 rows over 2 heads


def commit(L, s=None, caches=None, n=None, T=4, tl=FAKE, acc=1 << 21, al=1 << 22, seq=1 << 23,
           out=1 << 24, ws=FAKE, wsb=BIG):
    s = s or shape()
    caches = [cache()] if caches is None else caches
    arr = (_Cache * max(1, len(caches)))(*caches)
    return L.td_tree_commit(ctypes.byref(s), len(caches) if n is None else n, arr, T, tl, acc, al, seq,
                            out, ws, wsb, None)


def test_commit_refusals(L):
    assert commit(L, caches=[]) == INVALID
    assert commit(L, T=0) == INVALID and commit(L, T=129) == INVALID
    for name in ("acc", "al", "seq", "out", "ws"):
        assert commit(L, **{name: None}) == INVALID
    assert commit(L, tl=FAKE + 2) == INVALID
    assert commit(L, wsb=255) == WS_SMALL
    assert commit(L, out=1 << 23) == INVALID                 # new lengths over the old ones
    assert commit(L, out=(1 << 23) + 4) == INVALID
    assert commit(L, out=FAKE + 4) == INVALID                # over tree_lens
    assert commit(L, out=(1 << 21) + 28) == INVALID          # over accepted
    assert commit(L, caches=[cache(), cache(pages=3)]) == INVALID
    assert commit(L, caches=[cache(), cache(page=1001)]) == INVALID
    t = dict(page=16, blocks=63)
    assert commit(L, caches=[cache(table=FAKE, **t), cache(table=FAKE * 2, **t)]) == INVALID
    assert commit(L, caches=[cache(), cache(k=None)]) == INVALID


def append(L, s=None, c=None, n=5, k=FAKE, v=FAKE, stride=256, slots=FAKE):
    s, c = s or shape(), c or cache()
    return L.td_kv_append_slots(ctypes.byref(s), ctypes.byref(c), n, k, v, stride, slots, None)


def test_append_slots_refusals(L):
    assert append(L, n=-1) == INVALID
    assert append(L, k=None) == INVALID and append(L, v=FAKE + 8) == INVALID
    assert append(L, slots=None) == INVALID and append(L, slots=FAKE + 1) == INVALID
    assert append(L, stride=255) == INVALID and append(L, stride=260) == INVALID
    assert append(L, c=cache(k=None)) == INVALID
    assert append(L, s=shape(d=64)) == UNSUPPORTED
    assert append(L, n=0, k=None, v=None, slots=None) == 0    # nothing to do


TABLES = dict(B=3, page=16, blocks=8, pages=64, seq=1 << 20, new=1 << 21, table=1 << 22,
              held=1 << 23, held_out=1 << 24, free=1 << 25, count=1 << 26, count_out=1 << 27,
              cu=1 << 28, slots=1 << 29, max_new=10, ws=1 << 30, wsb=BIG)


def tables(L, **kw):
    a = dict(TABLES, **kw)
    return L.td_block_tables(a["B"], a["page"], a["blocks"], a["pages"], a["seq"], a["new"],
                             a["table"], a["held"], a["held_out"], a["free"], a["count"],
                             a["count_out"], a["cu"], a["slots"], a["max_new"], a["ws"], a["wsb"],
                             None)


def test_block_tables_refusals(L):
    for name in ("B", "page", "blocks", "pages"):
        assert tables(L, **{name: 0}) == INVALID
    assert tables(L, max_new=-1) == INVALID
    assert tables(L, B=65536) == UNSUPPORTED
    assert tables(L, blocks=1 << 27) == UNSUPPORTED
    assert tables(L, pages=1 << 27) == UNSUPPORTED
    assert tables(L, B=65535, blocks=1 << 16) == UNSUPPORTED
    for name in ("seq", "new", "table", "held", "held_out", "free", "count", "count_out", "cu",
                 "slots", "ws"):
        assert tables(L, **{name: None}) == INVALID
        assert tables(L, **{name: TABLES[name] + 2}) == INVALID
    assert tables(L, wsb=100) == WS_SMALL
    # overlapping arrays: only exactly in place, and only the two out pairs
    assert tables(L, held_out=TABLES["held"] + 4) == INVALID
    assert tables(L, held_out=TABLES["seq"]) == INVALID
    assert tables(L, cu=TABLES["new"] - 4) == INVALID
    assert tables(L, slots=TABLES["free"] + 252) == INVALID
    assert tables(L, count_out=TABLES["table"] + 92) == INVALID
    assert tables(L, count=TABLES["free"] + 252, count_out=TABLES["free"] + 252) == INVALID
