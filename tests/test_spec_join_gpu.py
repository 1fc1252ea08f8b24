"""Values that are not finite in results joined from the parts of several blocks."""
import pytest
import torch

from spec_util import D
from test_spec_gpu import _built, check_tree, run_tree, tree_case  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_a_value_that_is_not_finite_counts_at_any_probability(bad):
    """A drafted token whose score lies 200 below the context's, in a part of its own (one tile a
    block): a row that sees it gets its infinity, as softmax > 0 has it, whether or not the part's
    weight is a zero in fp32; rows that do not see it do not."""
    T, ctx = 2, 9088                              # 71 tiles of context, one of drafted tokens
    c = tree_case(3, 1, 1, [ctx + T], [T], T, 0, "empty")
    c["seen"][0, 0, 0] = True                     # row 0 sees token 0, row 1 none
    c["q"][:] = 1.0
    one = 100 * D ** -0.5                         # scores of +100 and -100
    c["K"][0, 0, :ctx] = one
    c["K"][0, 0, ctx:] = -one
    c["V"][0, 0, ctx, 9] = bad
    c["kc"], c["vc"] = c["K"], c["V"]
    out, ws = run_tree(c)
    got = out[0, :, 0].float().cpu()
    if bad != bad:
        assert torch.isnan(got[0, 9])
    else:
        assert got[0, 9] == bad
    clean = dict(c, V=c["V"].clone())
    clean["V"][0, 0, ctx, 9] = 0.0
    out[0, 0, 0, 9] = float(clean["V"][0, 0, :ctx, 9].double().mean())
    check_tree(clean, out)
    assert ws.status() == 0
