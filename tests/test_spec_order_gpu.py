"""Tree attention where a block takes several units of several tiles each: the
tensor-core work of a unit follows that of the unit before it."""
import pytest
import torch

from test_spec_gpu import _built, check_tree, run_tree, tree_case  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("page,k", [(0, 0), (16, 0), (64, 0), (0, 300), (16, 300)])
def test_many_units_of_several_tiles(page, k):
    """320 units of 2 to 5 tiles, 6 to 8 tiles a block: most units begin behind another one."""
    gen = torch.Generator().manual_seed(41 + page + k)
    B, T = 40, 3
    lens = torch.randint(260, 520, (B,), generator=gen).tolist()
    c = tree_case(page + k, 2, 8, lens, [T] * B, T, page, "tree", k, max_len=520)
    out, ws = run_tree(c)
    check_tree(c, out)
    assert ws.status() == 0
    for _ in range(3):
        assert torch.equal(run_tree(c, ws=ws)[0], out)


def test_units_of_one_and_of_several_tiles_in_turn():
    """Every order of one-tile and longer units next to each other in a block."""
    gen = torch.Generator().manual_seed(43)
    B, T = 160, 4
    lens = [T + int(n) for n in torch.randint(0, 400, (B,), generator=gen)]
    lens = [n if b % 3 else T + n % 100 for b, n in enumerate(lens)]
    c = tree_case(44, 4, 4, lens, [T] * B, T, 32, "tree", max_len=416)
    out, ws = run_tree(c)
    check_tree(c, out)
    assert ws.status() == 0
    assert torch.equal(run_tree(c, ws=ws)[0], out)
