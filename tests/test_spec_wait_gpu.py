"""Failure report of the tree attention's bounded waits.

The test switch "wait_test" makes the softmax warps wait on a barrier that
nothing arrives on, so their first wait runs out after "wait_limit_us": no
fault, no hang.  The CTA then waits (with limits) for the copies and products it
has in flight, reports TD_FLAG_WAIT_TIMEOUT and leaves; the next call on the same
workspace, with the switch off, is right."""
import pytest
import torch

import sparse_attention_td_gb300 as td
from test_spec_gpu import _built, check_tree, run_tree, tree_case  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [6, 60])
@pytest.mark.parametrize("page,k", [(0, 0), (16, 0), (24, 0), (0, 200)])
def test_wait_runs_out_then_the_next_call_is_right(T, page, k):
    c = tree_case(T + page, 4, 2, [900, 260], [T, T], T, page, "tree", k)
    out, ws = run_tree(c)
    check_tree(c, out)
    td.td_set_tuning("wait_limit_us", 20)
    td.td_set_tuning("wait_test", 1)
    try:
        run_tree(c, ws=ws)
    finally:
        td.td_set_tuning("wait_test", 0)
        td.td_set_tuning("wait_limit_us", 0)
    assert ws.status() == td.FLAG_WAIT_TIMEOUT
    again, _ = run_tree(c, ws=ws)
    assert ws.status() == 0
    assert torch.equal(again, out)
