"""Values that are not finite in small caches: what they cost, and whom they reach."""
import pytest
import torch

import sparse_attention_td_gb300 as td
from cache_util import D, U, attend
from test_cache_gpu import Case, _built, call, i32, near  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("q4", [False, True])
def test_rows_done_again_outlast_no_wait(q4):
    """Prompts between others whose every row sees a NaN: those rows are computed once more, one by one, and take
    far longer than a wait without progress may."""
    n, Hkv, G = 600, 8, 4
    c = Case(81, [n] * 8, G, Hkv, 0, q4)
    for b in (0, 2, 5, 6):
        if q4:
            c.parts[2][b, :, 3, 8:] = 0x7f
        else:
            c.parts[1][b, :, 3] = float("nan")
    q = 2 * c.rnd(8 * n, Hkv * G, D)
    out = torch.zeros_like(q).cuda()
    cu = i32([n * b for b in range(9)])
    td.td_set_tuning("wait_limit_us", 500)
    try:
        call(c)(c.shape, c.cache, 0, 0, cu, q.cuda(), c.seq, out, c.ws)
        torch.cuda.synchronize()
    finally:
        td.td_set_tuning("wait_limit_us", 0)
    assert c.ws.status() == 0
    sees = torch.ones(n, n, dtype=torch.bool).tril()
    for b in range(8):
        rows = slice(n * b, n * b + n)
        if b in (0, 2, 5, 6):
            assert out[rows][3:].isnan().all() and out[rows][:3].isfinite().all()
            continue
        for h in (0, 13, 31):
            ref, tol, _, _ = attend(q[rows, h], c.K[b, h // G], c.V[b, h // G], sees, 2.0 ** -11 if q4 else U, q4)
            near(out[rows, h], ref, tol)
