"""A tree call takes only a workspace with a part for tree calls, and the other calls
do not see that part (on the host: the library is a stand-in that counts calls)."""
import pytest
import torch

import sparse_attention_td_gb300 as td
from sparse_attention_td_gb300 import _lib
from sparse_attention_td_gb300 import build as libbuild

D = 128


@pytest.fixture
def calls(monkeypatch):
    """Workspaces in host memory; tree calls reach a stand-in instead of the library."""
    libbuild.build()
    real, seen = _lib.lib(), []

    class Stub:
        td_workspace_size = real.td_workspace_size
        td_tree_workspace_size = real.td_tree_workspace_size
        td_status_string = real.td_status_string

        @staticmethod
        def td_tree_attn(*a):
            seen.append(a)
            return 0

        td_tree_sparse_attn = td_tree_attn

    monkeypatch.setattr(_lib, "lib", lambda: Stub)
    monkeypatch.setattr(_lib, "td_workspace_init", lambda *a: None)
    monkeypatch.setattr(_lib, "_launch", lambda stream: (-1, 0))      # get_device() of a host tensor
    return seen


def attend(shape, T, ws, k=0):
    B, Hq, Hkv, N = shape.batch, shape.num_q_heads, shape.num_kv_heads, shape.max_seq_len
    q = torch.zeros(B, T, Hq, D, dtype=torch.bfloat16)
    cache = object.__new__(td.Cache)
    cache.ref, cache.fits = None, (-1, Hkv, None)
    lens = torch.zeros(B, dtype=torch.int32)
    if k:
        idx = torch.zeros(B, Hkv, k, dtype=torch.int32)
        td.td_tree_sparse_attn(shape, cache, T, None, None, q, lens, idx, k, torch.empty_like(q), ws)
    else:
        td.td_tree_attn(shape, cache, T, None, None, q, lens, torch.empty_like(q), ws)


@pytest.mark.parametrize("k", [0, 64])
def test_a_workspace_without_a_tree_part_is_refused(calls, k):
    shape = td.make_shape(4, 32, 8, 32768)
    ws = td.Workspace(shape, 64, device="cpu")
    assert ws.tensor.numel() > td.td_tree_workspace_size(shape, 16)      # large enough by its size
    with pytest.raises(ValueError, match="tree"):
        attend(shape, 16, ws, k)
    assert not calls


def test_a_tree_part_that_is_too_small_is_refused(calls):
    shape = td.make_shape(4, 32, 8, 32768)
    ws = td.Workspace(shape, 64, device="cpu", tree_size=4)
    for T in (1, 3, 4, 4):
        attend(shape, T, ws)
    assert len(calls) == 4
    with pytest.raises(ValueError, match="tree_size=16"):
        attend(shape, 16, ws)
    with pytest.raises(ValueError):
        attend(td.make_shape(4, 64, 8, 32768), 4, ws)                    # more query rows per KV head
    attend(td.make_shape(1, 8, 8, 100), 16, ws)                          # as many rows as 4 x G 4
    assert len(calls) == 5
    # beyond 128 rows per KV head a part of 128 rows serves every tree
    ws = td.Workspace(shape, 0, device="cpu", tree_size=32)
    attend(shape, 128, ws)


def test_the_other_calls_do_not_see_the_tree_part(calls):
    shape = td.make_shape(4, 32, 8, 32768)
    n, more = td.td_workspace_size(shape, 64), td.td_tree_workspace_size(shape, 16)
    ws = td.Workspace(shape, 64, device="cpu", tree_size=16)
    assert ws.nbytes == n and ws.tensor.numel() == n + more
    plain = td.Workspace(shape, 64, device="cpu")
    assert plain.nbytes == plain.tensor.numel() == n
